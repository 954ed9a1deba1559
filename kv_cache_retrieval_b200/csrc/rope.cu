// Rotary positions and the append to a paged key-value cache.
//
// y1 = m (x1 cos a - x2 sin a), y2 = m (x2 cos a + x1 sin a), a = pos * f_j, for the
// pairs (j, j + rot/2) or (2j, 2j+1) of a head; elements from rot on are copied.
//
// Both calls are one pass over memory: each element is read once and written
// once, a handful of float32 operations in between, so the bound is HBM (and
// the launch for a few tokens).  A thread owns one place in a head (2V
// elements: V pairs, or 2V copied ones) and walks over (token, head) rows with
// it, so its share of the angle table is read per row from shared memory; the
// table of the block's tokens is computed once per block, which divides the
// cost of the float64 angle and of sincospi by the number of heads.
//
// The angle: pos * f in turns is formed in float64 (an int32 position times a
// float64 frequency keeps 2^-53 relative, 1e-9 turns at 2^23 turns), reduced
// modulo one turn exactly (t - rint(t)) and only then rounded to float32 half
// turns for sincospif, so the float32 error is 2^-25 half turns at any
// position.

#include <algorithm>
#include <cstring>

#include "hhr_internal.cuh"
#include "paged_common.cuh"

namespace hhr {
namespace {

constexpr int kRopeThreads = 256;

struct RopeArgs {
  // rows to rotate in x's type: [T][H][d] (queries, or the tensor of hhr_rope)
  const void* x;
  void* y;
  int64_t x_tok, x_head, y_tok, y_head;
  int H, tail;                 // tail: elements from rot on have to be copied
  // keys and values of an append (Hkv == 0: none)
  const void* k;
  const void* v;
  void* K;
  void* V;
  int64_t k_row, v_row;
  int64_t k_page, k_head, k_tok, v_page, v_head, v_tok;
  float k_inv, v_inv;          // 1 / scale
  int Hkv;
  const int32_t* pos;
  const int32_t* rope_pos;     // nullable
  const int32_t* seq;          // nullable
  const int32_t* table;
  uint32_t* status;            // nullable
  int B, page, n_pages, table_cols, table_stride;
  const double* freqs;
  float mscale;
  int T, d, rot, interleaved;
  float sign;                  // -1 for the transposed rotation
  int heads;                   // H + 2 Hkv rows per token
  int rows_block;              // (token, head) rows per block
  int tokens_block;            // most tokens that a block's rows touch
  int places;                  // d / (2V) places of a head
};

template <typename T, int V>
__device__ __forceinline__ void load(const T* p, Pack<T, V>& r) {
  r = *reinterpret_cast<const Pack<T, V>*>(p);
}

// Converts and stores V elements; V = 8 to e4m3 is one 8-byte store.
template <typename TO, int V>
__device__ __forceinline__ void store(TO* p, const float (&f)[V], float mul) {
  Pack<TO, V> r;
#pragma unroll
  for (int e = 0; e < V; ++e) r.v[e] = from_f32<TO>(sizeof(TO) == 1 ? f[e] * mul : f[e]);
  *reinterpret_cast<Pack<TO, V>*>(p) = r;
}

// Where the pair (cos, sin) of element e of a place lies among the angles of a block: the 16-byte pieces (two pairs) of
// a place stand `turns` pieces apart, so that the places of a row read them from different banks.
template <int V>
__device__ __forceinline__ int angle_at(int t, int half, int turns, int place, int e) {
  return V == 1 ? 2 * (t * half + place) : 2 * t * half + ((e >> 1) * turns + place) * 4 + (e & 1) * 2;
}

// TI: type of x, y, k, v; TC: cache type; V: elements per access; U: rows a
// thread has in flight.
template <typename TI, typename TC, int V, int U>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int half = a.rot >> 1;
  float* cs = reinterpret_cast<float*>(smem);                             // [tokens_block][half] (cos, sin), see angle_at
  int64_t* slot = reinterpret_cast<int64_t*>(cs + static_cast<size_t>(a.tokens_block) * a.rot);  // K offset, V offset
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * a.rows_block;
  const int64_t rows_all = static_cast<int64_t>(a.T) * a.heads;
  const int rows = static_cast<int>(min(static_cast<int64_t>(a.rows_block), rows_all - row0));
  const int tok0 = static_cast<int>(static_cast<uint32_t>(row0) / static_cast<uint32_t>(a.heads));
  const int tok_n = static_cast<int>(static_cast<uint32_t>(row0 + rows - 1) / static_cast<uint32_t>(a.heads)) - tok0 + 1;

  const int I = a.places;
  const int place = threadIdx.x % I, first = threadIdx.x / I;
  const bool idle = first >= kRopeThreads / I;
  const bool turned = place * 2 * V < a.rot;
  // element places of the two halves of this thread's 2V elements
  const int p0 = turned && !a.interleaved ? place * V : place * 2 * V;
  const int p1 = turned && !a.interleaved ? half + place * V : place * 2 * V + V;
  const int turns = half / V;   // places that are turned

  dependency_wait();
  launch_dependents();

  // this thread's rows: U heads in a row, mostly of one token, all asked for before the angles are computed
  Pack<TI, V> x0[U], x1[U];
  int tok[U], head[U];
  bool live[U];
  {
    uint32_t row = static_cast<uint32_t>(row0) + static_cast<uint32_t>(min(first * U, rows - 1));
    int t = static_cast<int>(row / static_cast<uint32_t>(a.heads));
    int h = static_cast<int>(row - static_cast<uint32_t>(t) * static_cast<uint32_t>(a.heads));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      tok[u] = t;
      head[u] = h;
      live[u] = !idle && first * U + u < rows && (h >= a.H || turned || a.tail);
      if (live[u]) {
        const TI* p;
        if (h < a.H)
          p = static_cast<const TI*>(a.x) + t * a.x_tok + h * a.x_head;
        else if (h < a.H + a.Hkv)
          p = static_cast<const TI*>(a.k) + t * a.k_row + static_cast<int64_t>(h - a.H) * a.d;
        else
          p = static_cast<const TI*>(a.v) + t * a.v_row + static_cast<int64_t>(h - a.H - a.Hkv) * a.d;
        load<TI, V>(p + p0, x0[u]);
        load<TI, V>(p + p1, x1[u]);
      }
      if (++h == a.heads) {
        h = 0;
        ++t;
      }
    }
  }

  // the angles of the block's tokens
  for (int i = threadIdx.x; i < tok_n * half; i += kRopeThreads) {
    const int t = i / half, j = i - t * half;
    const int p = (a.rope_pos ? a.rope_pos : a.pos)[tok0 + t];
    const double turn = static_cast<double>(p) * a.freqs[j] * 0.15915494309189533577;
    const float r = static_cast<float>(2.0 * (turn - rint(turn)));
    float s, c;
    sincospif(r, &s, &c);
    *reinterpret_cast<float2*>(cs + angle_at<V>(t, half, turns, j / V, j % V)) = make_float2(a.mscale * c, a.sign * a.mscale * s);
  }
  // the places of the block's tokens in the cache: element offsets of K and V,
  // or -1 for a token that is not written
  if (a.Hkv) {
    for (int t = threadIdx.x; t < tok_n; t += kRopeThreads) {
      const int tok = tok0 + t, p = a.pos[tok], s = a.seq ? a.seq[tok] : tok;
      int64_t ko = -1, vo = -1;
      if (p >= 0) {
        const int col = p / a.page;
        int id = -1;
        if (s >= 0 && s < a.B && col < a.table_cols) id = a.table[static_cast<int64_t>(s) * a.table_stride + col];
        if (id >= 0 && id < a.n_pages) {
          ko = id * a.k_page + (p - col * a.page) * a.k_tok;
          vo = id * a.v_page + (p - col * a.page) * a.v_tok;
        } else if (a.status) {
          *a.status = HHR_ERR_BAD_INDEX;
        }
      }
      slot[2 * t] = ko;
      slot[2 * t + 1] = vo;
    }
  }
  __syncthreads();

  float w[2 * V];       // cosines and sines of this place, of token `have`
  int have = -1;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int t = tok[u] - tok0;
    if (!live[u] || (a.Hkv && slot[2 * t] < 0)) continue;
    const bool is_q = head[u] < a.H, is_v = head[u] >= a.H + a.Hkv;
    TI* yq = static_cast<TI*>(a.y) + tok[u] * a.y_tok + head[u] * a.y_head;
    TC* yc = is_v ? static_cast<TC*>(a.V) + slot[2 * t + 1] + (head[u] - a.H - a.Hkv) * a.v_head
                  : static_cast<TC*>(a.K) + slot[2 * t] + (head[u] - a.H) * a.k_head;
    if (is_v || !turned) {
      if (is_q) {
        *reinterpret_cast<Pack<TI, V>*>(yq + p0) = x0[u];
        *reinterpret_cast<Pack<TI, V>*>(yq + p1) = x1[u];
      } else if constexpr (sizeof(TC) == sizeof(TI)) {   // the same type: the bits as they are
        *reinterpret_cast<Pack<TI, V>*>(yc + p0) = x0[u];
        *reinterpret_cast<Pack<TI, V>*>(yc + p1) = x1[u];
      }
      if constexpr (sizeof(TC) != sizeof(TI)) {
        if (!is_q) {
          float f0[V], f1[V];
#pragma unroll
          for (int e = 0; e < V; ++e) {
            f0[e] = to_f32(x0[u].v[e]);
            f1[e] = to_f32(x1[u].v[e]);
          }
          store<TC, V>(yc + p0, f0, is_v ? a.v_inv : a.k_inv);
          store<TC, V>(yc + p1, f1, is_v ? a.v_inv : a.k_inv);
        }
      }
      continue;
    }
    if (have != t) {
      have = t;
      if constexpr (V == 1) {
        const float2 z = *reinterpret_cast<const float2*>(cs + angle_at<V>(t, half, turns, place, 0));
        w[0] = z.x;
        w[1] = z.y;
      } else {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const float4 z = *reinterpret_cast<const float4*>(cs + angle_at<V>(t, half, turns, place, e));
          w[2 * e] = z.x;
          w[2 * e + 1] = z.y;
          w[2 * e + 2] = z.z;
          w[2 * e + 3] = z.w;
        }
      }
    }
    float f0[V], f1[V];
    if (a.interleaved) {
      float g[2 * V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        g[e] = to_f32(x0[u].v[e]);
        g[V + e] = to_f32(x1[u].v[e]);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float u1 = g[2 * e], u2 = g[2 * e + 1];
        g[2 * e] = fmaf(u1, w[2 * e], -(u2 * w[2 * e + 1]));
        g[2 * e + 1] = fmaf(u2, w[2 * e], u1 * w[2 * e + 1]);
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        f0[e] = g[e];
        f1[e] = g[V + e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float u1 = to_f32(x0[u].v[e]), u2 = to_f32(x1[u].v[e]);
        f0[e] = fmaf(u1, w[2 * e], -(u2 * w[2 * e + 1]));
        f1[e] = fmaf(u2, w[2 * e], u1 * w[2 * e + 1]);
      }
    }
    if (is_q) {
      store<TI, V>(yq + p0, f0, 1.0f);
      store<TI, V>(yq + p1, f1, 1.0f);
    } else {
      store<TC, V>(yc + p0, f0, a.k_inv);
      store<TC, V>(yc + p1, f1, a.k_inv);
    }
  }
}

// The accesses of a launch are 16 bytes wide where every row, and every place
// in a row, starts on 16 bytes (8 on the 8-bit side of an append); otherwise
// they go element by element.
template <typename TI, typename TC, int V>
cudaError_t launch_rows(RopeArgs& a, cudaStream_t stream) {
  a.places = a.d / (2 * V);
  const int step = kRopeThreads / a.places;
  const int64_t rows = static_cast<int64_t>(a.T) * a.heads;
  const int U = rows >= static_cast<int64_t>(step) * 4 * 592 ? 4 : 1;
  a.rows_block = step * U;
  a.tokens_block = std::min(a.rows_block, (a.rows_block - 2) / a.heads + 2);
  const size_t smem = static_cast<size_t>(a.tokens_block) * ((a.rot >> 1) * sizeof(float2) + 2 * sizeof(int64_t));
  const dim3 grid(static_cast<unsigned>((rows + a.rows_block - 1) / a.rows_block));
  static std::atomic<size_t> raised[2][kMaxDevices];
  auto kern = U == 4 ? rope_kernel<TI, TC, V, 4> : rope_kernel<TI, TC, V, 1>;
  if (smem > 48 * 1024)
    if (cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), smem, raised[U == 4])) return e;
  return launch_dependent<RopeArgs>(kern, grid, kRopeThreads, smem, stream, a);
}

template <typename TI, typename TC>
cudaError_t launch_typed(RopeArgs& a, bool wide, cudaStream_t stream) {
  return wide ? launch_rows<TI, TC, 16 / sizeof(TI)>(a, stream) : launch_rows<TI, TC, 1>(a, stream);
}

int32_t check_rotation(const hhr_rotation* r, const double* freqs, int d) {
  if (r->rot < 0 || r->rot > d || (r->rot & 1)) return HHR_ERR_INVALID_ARG;
  if (r->flags & ~(HHR_ROPE_INTERLEAVED | HHR_ROPE_TRANSPOSE)) return HHR_ERR_INVALID_ARG;
  if (!std::isfinite(r->mscale)) return HHR_ERR_INVALID_ARG;
  if (r->rot > 0 && (!freqs || !aligned_to(freqs, 8))) return HHR_ERR_INVALID_ARG;
  return HHR_OK;
}

bool wide_row(const void* p, int64_t tok, int64_t head, int size) {
  return aligned_to(p, 16) && (tok * size) % 16 == 0 && (head * size) % 16 == 0;
}

// Whether rows of d elements at t * s + h * u (t < m, h < n) may share elements:
// the wider of the two strides has to step over all rows of the narrower one.
bool rows_overlap(int64_t m, int64_t s, int64_t n, int64_t u, int64_t d) {
  if (m == 1) return n > 1 && u < d;
  if (n == 1) return s < d;
  return s <= u ? s < d || u < (m - 1) * s + d : u < d || s < (n - 1) * u + d;
}

int32_t status_of(cudaError_t e) { return e == cudaSuccess ? HHR_OK : HHR_ERR_CUDA; }

}  // namespace
}  // namespace hhr

using namespace hhr;

extern "C" {

int32_t hhr_rope_freqs(const hhr_rope_scaling* s, int32_t rot, double* freqs, float* mscale) {
  if (!s || !freqs || !mscale || rot < 2 || (rot & 1)) return HHR_ERR_INVALID_ARG;
  if (!(s->base > 1) || !std::isfinite(s->base)) return HHR_ERR_INVALID_ARG;
  if (s->kind < HHR_ROPE_SCALE_NONE || s->kind > HHR_ROPE_SCALE_BANDS) return HHR_ERR_INVALID_ARG;
  if (s->kind != HHR_ROPE_SCALE_NONE && (!(s->factor >= 1) || !std::isfinite(s->factor))) return HHR_ERR_INVALID_ARG;
  const bool ramp = s->kind == HHR_ROPE_SCALE_YARN || s->kind == HHR_ROPE_SCALE_BANDS;
  if (ramp && (s->orig < 1 || !(s->low > 0) || !(s->high > s->low) || !std::isfinite(s->high))) return HHR_ERR_INVALID_ARG;
  if (s->kind == HHR_ROPE_SCALE_NTK && rot == 2) return HHR_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925;
  const int half = rot / 2;
  double base = s->base;
  if (s->kind == HHR_ROPE_SCALE_NTK) base *= std::pow(s->factor, rot / (rot - 2.0));
  double lo = 0, hi = 0;
  if (s->kind == HHR_ROPE_SCALE_YARN) {
    const auto dim = [&](double turns) { return rot * std::log(s->orig / (two_pi * turns)) / (2 * std::log(base)); };
    lo = std::max(std::floor(dim(s->high)), 0.0);
    hi = std::min(std::ceil(dim(s->low)), half - 1.0);
  }
  for (int j = 0; j < half; ++j) {
    double f = std::pow(base, -2.0 * j / rot);
    if (s->kind == HHR_ROPE_SCALE_LINEAR) f /= s->factor;
    if (s->kind == HHR_ROPE_SCALE_YARN) {
      const double w = std::min(std::max((j - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
      f = f * (1 - w) + f / s->factor * w;
    }
    if (s->kind == HHR_ROPE_SCALE_BANDS) {
      const double w = std::min(std::max((s->orig * f / two_pi - s->low) / (s->high - s->low), 0.0), 1.0);
      f = f / s->factor * (1 - w) + f * w;
    }
    freqs[j] = f;
  }
  *mscale = s->kind == HHR_ROPE_SCALE_YARN ? static_cast<float>(0.1 * std::log(s->factor) + 1.0) : 1.0f;
  return HHR_OK;
}

int32_t hhr_rope(int32_t T, int32_t H, int32_t d, int32_t type, const hhr_rotation* rotation,
                 const double* freqs, const int32_t* pos, const void* x, int64_t x_tok,
                 int64_t x_head, void* y, int64_t y_tok, int64_t y_head, void* stream) {
  if (T < 0 || H < 0 || d < 2 || (d & 1) || !rotation) return HHR_ERR_INVALID_ARG;
  if (type != HHR_TYPE_BF16 && type != HHR_TYPE_F16 && type != HHR_TYPE_F32) return HHR_ERR_INVALID_ARG;
  if (int32_t st = check_rotation(rotation, freqs, d)) return st;
  if (x_tok < 0 || x_head < 0 || y_tok < 0 || y_head < 0) return HHR_ERR_INVALID_ARG;
  if (d > 512 || static_cast<int64_t>(T) * H >= (int64_t{1} << 31)) return HHR_ERR_UNSUPPORTED;
  if (T == 0 || H == 0) return HHR_OK;
  const int size = type_size(type);
  if (!pos || !aligned_to(pos, 4) || !x || !y || !aligned_to(x, size) || !aligned_to(y, size)) return HHR_ERR_INVALID_ARG;
  if (rows_overlap(T, y_tok, H, y_head, d)) return HHR_ERR_INVALID_ARG;
  if (x == y && ((T > 1 && x_tok != y_tok) || (H > 1 && x_head != y_head))) return HHR_ERR_INVALID_ARG;
  RopeArgs a;
  std::memset(&a, 0, sizeof a);
  a.x = x;
  a.y = y;
  a.x_tok = x_tok;
  a.x_head = x_head;
  a.y_tok = y_tok;
  a.y_head = y_head;
  a.H = a.heads = H;
  a.tail = x != y;
  a.pos = pos;
  a.freqs = freqs;
  a.mscale = rotation->mscale;
  a.sign = (rotation->flags & HHR_ROPE_TRANSPOSE) ? -1.0f : 1.0f;
  a.interleaved = (rotation->flags & HHR_ROPE_INTERLEAVED) ? 1 : 0;
  a.T = T;
  a.d = d;
  a.rot = rotation->rot;
  const int unit = 32 / size;   // two accesses of 16 bytes
  const bool wide = d % unit == 0 && a.rot % unit == 0 && wide_row(x, x_tok, x_head, size) && wide_row(y, y_tok, y_head, size);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (type) {
    case HHR_TYPE_BF16: return status_of(launch_typed<__nv_bfloat16, __nv_bfloat16>(a, wide, s));
    case HHR_TYPE_F16: return status_of(launch_typed<__half, __half>(a, wide, s));
    default: return status_of(launch_typed<float, float>(a, wide, s));
  }
}

int32_t hhr_paged_append(const hhr_paged* cache, int32_t T, int32_t B,
                         const hhr_rotation* rotation, const double* freqs, const int32_t* pos,
                         const int32_t* rope_pos, const int32_t* seq, const int32_t* table,
                         const void* q, int64_t q_tok, void* q_out, int64_t q_out_tok,
                         const void* k, int64_t k_row, const void* v, int64_t v_row, void* K,
                         void* V, uint32_t* status, void* stream) {
  if (int32_t st = check_paged(cache)) return st;
  const hhr_paged& c = *cache;
  if (T < 0 || B < 0 || (q == nullptr) != (q_out == nullptr)) return HHR_ERR_INVALID_ARG;
  if (rotation) {
    if (rotation->flags & HHR_ROPE_TRANSPOSE) return HHR_ERR_INVALID_ARG;
    if (int32_t st = check_rotation(rotation, freqs, c.d)) return st;
  }
  const int64_t q_width = static_cast<int64_t>(c.Hq) * c.d;
  if (T > 1 && (k_row < 0 || v_row < 0 || (q && (q_tok < 0 || q_out_tok < q_width)))) return HHR_ERR_INVALID_ARG;
  if (q && q == q_out && T > 1 && q_tok != q_out_tok) return HHR_ERR_INVALID_ARG;
  if (!seq && T > B) return HHR_ERR_INVALID_ARG;
  if (static_cast<int64_t>(T) * (c.Hq + 2 * static_cast<int64_t>(c.Hkv)) >= (int64_t{1} << 31)) return HHR_ERR_UNSUPPORTED;
  if (T == 0) return HHR_OK;
  if (!pos || !table || !k || !v || !K || !V) return HHR_ERR_INVALID_ARG;
  if (!aligned_to(K, 16) || !aligned_to(V, 16) || !aligned_to(pos, 4) || !aligned_to(table, 4) || !aligned_to(rope_pos, 4) ||
      !aligned_to(seq, 4) || !aligned_to(status, 4) || !aligned_to(k, 2) || !aligned_to(v, 2) || !aligned_to(q, 2) ||
      !aligned_to(q_out, 2))
    return HHR_ERR_INVALID_ARG;
  RopeArgs a;
  std::memset(&a, 0, sizeof a);
  a.x = q;
  a.y = q_out;
  a.x_tok = q_tok;
  a.y_tok = q_out_tok;
  a.x_head = a.y_head = c.d;
  a.H = q ? c.Hq : 0;
  a.tail = q != q_out;
  a.k = k;
  a.v = v;
  a.K = K;
  a.V = V;
  a.k_row = k_row;
  a.v_row = v_row;
  a.k_page = c.k_page;
  a.k_head = c.k_head;
  a.k_tok = c.k_tok;
  a.v_page = c.v_page;
  a.v_head = c.v_head;
  a.v_tok = c.v_tok;
  a.k_inv = 1.0f / c.k_scale;
  a.v_inv = 1.0f / c.v_scale;
  a.Hkv = c.Hkv;
  a.pos = pos;
  a.rope_pos = rope_pos;
  a.seq = seq;
  a.table = table;
  a.status = status;
  a.B = B;
  a.page = c.page;
  a.n_pages = c.n_pages;
  a.table_cols = c.table_cols;
  a.table_stride = c.table_stride;
  a.freqs = freqs;
  a.mscale = rotation ? rotation->mscale : 1.0f;
  a.sign = 1.0f;
  a.interleaved = rotation && (rotation->flags & HHR_ROPE_INTERLEAVED) ? 1 : 0;
  a.T = T;
  a.d = c.d;
  a.rot = rotation ? rotation->rot : 0;
  a.heads = a.H + 2 * c.Hkv;
  const bool wide = a.rot % 16 == 0 && wide_row(k, k_row, 0, 2) && wide_row(v, v_row, 0, 2) &&
                    (!q || (wide_row(q, q_tok, 0, 2) && wide_row(q_out, q_out_tok, 0, 2)));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool e4m3 = c.kv_type == HHR_TYPE_E4M3;
  if (c.q_type == HHR_TYPE_BF16)
    return status_of(e4m3 ? launch_typed<__nv_bfloat16, __nv_fp8_e4m3>(a, wide, s)
                          : launch_typed<__nv_bfloat16, __nv_bfloat16>(a, wide, s));
  return status_of(e4m3 ? launch_typed<__half, __nv_fp8_e4m3>(a, wide, s) : launch_typed<__half, __half>(a, wide, s));
}

}  // extern "C"
