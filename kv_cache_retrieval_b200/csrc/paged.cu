// Attention of one new token per sequence over a paged key-value cache.
//
// One CTA per (sequence, query head): its warps take the tokens in turn, each
// with its own running maximum, sum and output (float32), merged at the end
// in the order of the warps.

#include <algorithm>
#include <cfloat>
#include <cstring>

#include "hhr_internal.cuh"
#include "paged_common.cuh"

namespace hhr {
namespace {

constexpr int kPagedThreads = 256;
constexpr int kPagedWarps = kPagedThreads / 32;

struct PagedArgs {
  const void* q;
  const void* K;
  const void* V;
  const int32_t* table;
  const int32_t* lens;
  void* out;
  float* lse;
  uint32_t* status;
  int64_t q_seq, k_page, k_head, k_tok, v_page, v_head, v_tok;
  float scale_log2, v_scale;
  int B, Hq, Hkv, page, n_pages, table_cols, table_stride, window, out_f32;
};

template <typename TQ, typename TC, int D>
__global__ void __launch_bounds__(kPagedThreads) paged_kernel(const PagedArgs a) {
  constexpr int E = D / 32;
  __shared__ float s_m[kPagedWarps], s_l[kPagedWarps], s_o[kPagedWarps][D];
  const int b = blockIdx.x / a.Hq, h = blockIdx.x % a.Hq, g = h / (a.Hq / a.Hkv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  dependency_wait();
  launch_dependents();
  int len = a.lens[b];
  if (len < 0 || len > static_cast<int64_t>(a.table_cols) * a.page) {
    if (threadIdx.x == 0) *a.status = HHR_ERR_BAD_INDEX;
    len = 0;
  }
  const int lo = a.window ? max(0, len - a.window) : 0;
  float q[E], o[E], m = -INFINITY, l = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = to_f32(static_cast<const TQ*>(a.q)[b * a.q_seq + h * D + e * 32 + lane]);
    o[e] = 0;
  }
  for (int n = lo + warp; n < len; n += kPagedWarps) {
    const int id = a.table[static_cast<int64_t>(b) * a.table_stride + n / a.page];
    if (id < 0 || id >= a.n_pages) {
      *a.status = HHR_ERR_BAD_INDEX;
      continue;
    }
    const TC* k = static_cast<const TC*>(a.K) + id * a.k_page + g * a.k_head + (n % a.page) * a.k_tok;
    const TC* v = static_cast<const TC*>(a.V) + id * a.v_page + g * a.v_head + (n % a.page) * a.v_tok;
    float x = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) x = fmaf(q[e], to_f32(k[e * 32 + lane]), x);
#pragma unroll
    for (int w = 16; w; w >>= 1) x += __shfl_xor_sync(~0u, x, w);
    x *= a.scale_log2;
    const float mn = fmaxf(m, x), base = mn == -INFINITY ? 0.0f : mn;
    const float c = exp2f(m - base), p = exp2f(x - base);
    m = mn;
    l = l * c + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], c, p * to_f32(v[e * 32 + lane]));
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][e * 32 + lane] = o[e];
  __syncthreads();
  float M = -INFINITY, L = 0;
  for (int w = 0; w < kPagedWarps; ++w) M = fmaxf(M, s_m[w]);
  const float base = M == -INFINITY ? 0.0f : M;
  for (int w = 0; w < kPagedWarps; ++w) L += s_l[w] * exp2f(s_m[w] - base);
  const float inv = L > 0 ? a.v_scale / L : (L == 0 ? 0.0f : L);
  for (int e = threadIdx.x; e < D; e += kPagedThreads) {
    float y = 0;
    for (int w = 0; w < kPagedWarps; ++w) y += s_o[w][e] * exp2f(s_m[w] - base);
    y *= inv;
    const size_t at = (static_cast<size_t>(b) * a.Hq + h) * D + e;
    if (a.out_f32)
      static_cast<float*>(a.out)[at] = y;
    else
      static_cast<TQ*>(a.out)[at] = from_f32<TQ>(y);
  }
  if (threadIdx.x == 0 && a.lse)
    a.lse[static_cast<size_t>(b) * a.Hq + h] = L == 0 ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
}

template <typename TQ, typename TC>
cudaError_t launch_paged(const PagedArgs& a, int d, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.B) * a.Hq);
  switch (d) {
    case 64: return launch_dependent<PagedArgs>(paged_kernel<TQ, TC, 64>, grid, kPagedThreads, 0, s, a);
    case 128: return launch_dependent<PagedArgs>(paged_kernel<TQ, TC, 128>, grid, kPagedThreads, 0, s, a);
    default: return launch_dependent<PagedArgs>(paged_kernel<TQ, TC, 256>, grid, kPagedThreads, 0, s, a);
  }
}

}  // namespace
}  // namespace hhr

using namespace hhr;

extern "C" {

size_t hhr_paged_workspace_size(const hhr_paged* cache) { return check_paged(cache) == HHR_OK ? 256 : 0; }

int32_t hhr_paged_attend(const hhr_paged* cache, int32_t B, const void* q, int64_t q_seq,
                         const void* K, const void* V, const int32_t* table, const int32_t* lens,
                         int32_t window, float scale, int32_t out_type, void* out, float* lse,
                         void* workspace, size_t ws_bytes, void* stream) {
  if (int32_t st = check_paged(cache)) return st;
  const hhr_paged& c = *cache;
  if (B < 0 || window < 0 || !std::isfinite(scale)) return HHR_ERR_INVALID_ARG;
  if (out_type != c.q_type && out_type != HHR_TYPE_F32) return HHR_ERR_INVALID_ARG;
  if (static_cast<int64_t>(B) * c.Hq >= (int64_t{1} << 31)) return HHR_ERR_UNSUPPORTED;
  if (!workspace || !aligned_to(workspace, 256) || ws_bytes < hhr_paged_workspace_size(cache)) return HHR_ERR_WORKSPACE;
  if (B == 0) return HHR_OK;
  if (!q || !K || !V || !table || !lens || !out) return HHR_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(K, 16) || !aligned_to(V, 16) || !aligned_to(out, 16) || !aligned_to(table, 4) ||
      !aligned_to(lens, 4) || !aligned_to(lse, 4))
    return HHR_ERR_INVALID_ARG;
  if (B > 1 && (q_seq < 0 || q_seq % 8 != 0)) return HHR_ERR_INVALID_ARG;
  PagedArgs a;
  std::memset(&a, 0, sizeof a);
  a.q = q;
  a.K = K;
  a.V = V;
  a.table = table;
  a.lens = lens;
  a.out = out;
  a.lse = lse;
  a.status = static_cast<uint32_t*>(workspace);
  a.q_seq = q_seq;
  a.k_page = c.k_page;
  a.k_head = c.k_head;
  a.k_tok = c.k_tok;
  a.v_page = c.v_page;
  a.v_head = c.v_head;
  a.v_tok = c.v_tok;
  a.scale_log2 = scale * c.k_scale * 1.4426950408889634f;
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
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (c.q_type == HHR_TYPE_BF16)
    e = c.kv_type == HHR_TYPE_E4M3 ? launch_paged<__nv_bfloat16, __nv_fp8_e4m3>(a, c.d, s)
                                   : launch_paged<__nv_bfloat16, __nv_bfloat16>(a, c.d, s);
  else
    e = c.kv_type == HHR_TYPE_E4M3 ? launch_paged<__half, __nv_fp8_e4m3>(a, c.d, s)
                                   : launch_paged<__half, __half>(a, c.d, s);
  return e == cudaSuccess ? HHR_OK : HHR_ERR_CUDA;
}

}  // extern "C"
