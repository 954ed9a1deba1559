"""ensure_smem_limit (csrc/hhr_internal.cuh) against a fake of the CUDA calls, compiled for the host."""
import ctypes as C
import os
import subprocess

from kv_cache_retrieval_b200 import build as kbuild

SOURCE = r"""
#include <condition_variable>
#include <chrono>
#include <thread>
#include "hhr_internal.cuh"

static std::mutex m;
static std::condition_variable cv;
static int limit = 0, device = 0, calls = 0;
static bool small_called = false, large_set = false;
static cudaError_t answer = cudaSuccess;

extern "C" cudaError_t CUDARTAPI cudaGetDevice(int* dev) {
  *dev = device;
  return cudaSuccess;
}
// The smaller size is set as late as it can be: behind the larger one, or after a while if nothing lets that through.
extern "C" cudaError_t CUDARTAPI cudaFuncSetAttribute(const void*, cudaFuncAttribute, int bytes) {
  std::unique_lock<std::mutex> lock(m);
  ++calls;
  if (answer != cudaSuccess) return answer;
  if (bytes == 1000) {
    small_called = true;
    cv.notify_all();
    cv.wait_for(lock, std::chrono::milliseconds(500), [] { return large_set; });
  }
  limit = bytes;
  if (bytes == 2000) {
    large_set = true;
    cv.notify_all();
  }
  return cudaSuccess;
}

static std::atomic<size_t> record[hhr::kMaxDevices];

extern "C" int two_first_calls(int* kept) {
  std::thread a([] { hhr::ensure_smem_limit(nullptr, 1000, record); });
  std::thread b([] {
    {
      std::unique_lock<std::mutex> lock(m);
      cv.wait(lock, [] { return small_called; });
    }
    hhr::ensure_smem_limit(nullptr, 2000, record);
  });
  a.join();
  b.join();
  *kept = static_cast<int>(record[0].load());
  return limit;
}
extern "C" int one_call(int dev, int bytes, int fail) {
  device = dev;
  answer = fail ? cudaErrorInvalidValue : cudaSuccess;
  return hhr::ensure_smem_limit(nullptr, bytes, record);
}
extern "C" int attribute_calls() { return calls; }
"""


def load(tmp_path):
    src, lib = tmp_path / "smem.cpp", tmp_path / "smem.so"
    src.write_text(SOURCE)
    cuda = os.path.dirname(os.path.dirname(kbuild._nvcc())) or "/usr/local/cuda"
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I", kbuild.CSRC, "-I",
                    kbuild.INCLUDE, "-I", os.path.join(cuda, "include"), str(src), "-o", str(lib)], check=True)
    return C.CDLL(str(lib))


def test_the_larger_of_two_threads_first_sizes_stays(tmp_path):
    kept = C.c_int()
    assert load(tmp_path).two_first_calls(C.byref(kept)) >= kept.value == 2000


def test_set_once_per_size_and_device_and_again_after_a_failure(tmp_path):
    lib = load(tmp_path)
    for dev, bytes_, fail, status, calls in [(0, 50000, 1, 1, 1), (0, 50000, 0, 0, 2), (0, 50000, 0, 0, 2), (0, 40000, 0, 0, 2),
                                             (0, 60000, 0, 0, 3), (1, 40000, 0, 0, 4), (1, 40000, 0, 0, 4),
                                             (70, 40000, 0, 0, 5), (70, 40000, 0, 0, 6)]:
        assert lib.one_call(dev, bytes_, fail) == status
        assert lib.attribute_calls() == calls
