// hhr_paged_attend: checks, workspace and launch (the kernel: paged_attend.cuh).

#include <cstring>

#include "paged_attend.cuh"

namespace hhr {
namespace {

// Workspace: status word, counters, exchanged states.
constexpr size_t kPagedCounters = 256;
constexpr size_t kPagedParts = kPagedCounters + (kPagedMaxGrid * sizeof(uint32_t) + 255) / 256 * 256;

// Query heads of a unit: the heads of a KV head in equal chunks of at most paged_max_heads.
int unit_chunks(const hhr_paged& c) { return (c.Hq / c.Hkv + paged_max_heads(c.d) - 1) / paged_max_heads(c.d); }
int unit_heads(const hhr_paged& c) { return (c.Hq / c.Hkv + unit_chunks(c) - 1) / unit_chunks(c); }

}  // namespace
}  // namespace hhr

using namespace hhr;

extern "C" {

size_t hhr_paged_workspace_size(const hhr_paged* cache) {
  if (check_paged(cache) != HHR_OK) return 0;
  const size_t state = paged_state(unit_heads(*cache), cache->d);
  return align_up(kPagedParts + (2 + kPagedMaxWarps) * kPagedMaxGrid * state * sizeof(float), 256);
}

int32_t hhr_paged_attend(const hhr_paged* cache, int32_t B, const void* q, int64_t q_seq,
                         const void* K, const void* V, const int32_t* table, const int32_t* lens,
                         int32_t window, float scale, int32_t out_type, void* out, float* lse,
                         void* workspace, size_t ws_bytes, void* stream) {
  if (int32_t st = check_paged(cache)) return st;
  const hhr_paged& c = *cache;
  const float scale_log2 = std::fabs(scale) * c.k_scale * 1.4426950408889634f;
  if (B < 0 || window < 0 || !std::isfinite(scale_log2)) return HHR_ERR_INVALID_ARG;
  if (out_type != c.q_type && out_type != HHR_TYPE_F32) return HHR_ERR_INVALID_ARG;
  if (static_cast<int64_t>(B) * c.Hq >= (int64_t{1} << 31)) return HHR_ERR_UNSUPPORTED;
  // a warp's tiles are counted in 32 bits
  if (static_cast<double>(B) * c.Hq * (static_cast<double>(c.table_cols) * c.page / 16 + 1) >= 0x1p36) return HHR_ERR_UNSUPPORTED;
  if (!workspace || !aligned_to(workspace, 256) || ws_bytes < hhr_paged_workspace_size(cache)) return HHR_ERR_WORKSPACE;
  if (B == 0) return HHR_OK;
  if (!q || !K || !V || !table || !lens || !out) return HHR_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(K, 16) || !aligned_to(V, 16) || !aligned_to(out, 16) || !aligned_to(table, 4) ||
      !aligned_to(lens, 4) || !aligned_to(lse, 4))
    return HHR_ERR_INVALID_ARG;
  if (B > 1 && (q_seq < 0 || q_seq % 8 != 0)) return HHR_ERR_INVALID_ARG;
  const int size = type_size(c.kv_type);
  PagedArgs a;
  std::memset(&a, 0, sizeof a);
  a.q = q;
  a.K = K;
  a.V = V;
  a.table = table;
  a.lens = lens;
  a.out = out;
  a.lse = lse;
  char* const ws = static_cast<char*>(workspace);
  a.status = reinterpret_cast<uint32_t*>(ws);
  a.counters = reinterpret_cast<uint32_t*>(ws + kPagedCounters);
  a.parts = reinterpret_cast<float*>(ws + kPagedParts);
  a.q_seq = q_seq;
  a.k_page = c.k_page * size;
  a.k_head = c.k_head * size;
  a.k_tok = c.k_tok * size;
  a.v_page = c.v_page * size;
  a.v_head = c.v_head * size;
  a.v_tok = c.v_tok * size;
  a.scale_log2 = scale_log2;
  a.flip = scale < 0 ? 0x80008000u : 0;
  a.v_scale = c.v_scale;
  a.B = B;
  a.Hq = c.Hq;
  a.Hkv = c.Hkv;
  a.page = c.page;
  a.n_pages = c.n_pages;
  a.table_cols = c.table_cols;
  a.table_stride = c.table_stride;
  a.window = window;
  a.out_f32 = out_type == HHR_TYPE_F32;
  a.r = c.Hq / c.Hkv;
  a.chunk = unit_heads(c);
  a.chunks = unit_chunks(c);
  a.state = paged_state(a.chunk, c.d);
  a.firsts = a.parts + static_cast<size_t>(2 * kPagedMaxGrid) * a.state;
  while ((int64_t{1} << a.page_shift) < c.page) ++a.page_shift;
  a.page_magic = static_cast<uint32_t>((((uint64_t{1} << a.page_shift) - c.page) << 32) / c.page + 1);
  a.min_tiles = 2;   // 517 tokens, 8 KV heads: 9.6 us; with 1 (more CTAs that share a unit) 13.6
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return HHR_ERR_CUDA;
  const int grid = std::min(sms, kPagedMaxGrid);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool e4m3 = c.kv_type == HHR_TYPE_E4M3;
  cudaError_t e;
  if (c.q_type == HHR_TYPE_BF16)
    e = e4m3 ? launch_paged_bf16_e4m3(a, c.d, grid, s) : launch_paged_bf16(a, c.d, grid, s);
  else
    e = e4m3 ? launch_paged_f16_e4m3(a, c.d, grid, s) : launch_paged_f16(a, c.d, grid, s);
  return e == cudaSuccess ? HHR_OK : HHR_ERR_CUDA;
}

}  // extern "C"
