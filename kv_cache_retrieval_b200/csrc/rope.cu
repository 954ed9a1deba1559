// Rotary positions and the append to a paged key-value cache.
//
// y1 = m (x1 cos a - x2 sin a), y2 = m (x2 cos a + x1 sin a), a = pos * f_j, for the
// pairs (j, j + rot/2) or (2j, 2j+1) of a head; elements from rot on are copied.
//
// Both calls are one pass over memory: each element is read once and written
// once, a handful of float32 operations in between, so the bound is HBM (and
// the launch for a few tokens).  A thread owns one place in a head (2V
// elements: V pairs, or 2V copied ones) and U heads of one token with it, whose
// pairs turn by the same V angles.  The angles of a tile's tokens are computed
// once, for all of their heads, while rows are on their way.
//
// Measured (B200): 8192 tokens x 40 heads of 128, bf16: 29.5 us, 5.7 TB/s (0.88
// of the copy bandwidth); float32, half of each head, pairs interleaved, 4095 x 32
// heads: 24.5 us, 5.5 TB/s; append of 8191 tokens (32 + 2 x 8 heads of 128, fp16):
// 36.3 us, 5.6 TB/s.  Without the angles they take the same time.
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
  int places;                  // d / (2V) places of a head
  int q_groups, kv_groups, groups;   // groups of heads: of queries, of keys (and of values), of a token
  uint32_t units;
  int tiles;                   // (token, group) pairs, and tiles of as many as a block has rows of threads
  int tokens_block;            // most tokens that a tile touches
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

// What a thread has of a tile (as many (token, group of U heads) as a block has rows of threads).
struct RopePart {
  int tok0, tok_n;   // the tile's tokens
  int t;             // the thread's token of these
  int kind;          // 0 queries, 1 keys, 2 values
  int head, n;       // its first head and how many
};

// TI: type of x, y, k, v; TC: cache type; V: elements per access; U: heads of a token that a thread takes; kCache: keys
// and values go to a cache.
template <typename TI, typename TC, int V, int U, bool kCache>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
  constexpr bool kStaged = V > 1 && U > 1;   // rows come through shared memory, a tile ahead; or else by plain loads
  extern __shared__ __align__(16) unsigned char smem[];
  const int half = a.rot >> 1;
  // two tiles' rows, [2][U][2][threads] accesses; two tiles' (cos, sin), see angle_at; their K and V offsets
  Pack<TI, V>* const rows = reinterpret_cast<Pack<TI, V>*>(smem);
  float* const cs_all = reinterpret_cast<float*>(smem + (kStaged ? 2 * U * 2 * kRopeThreads * 16 : 0));
  int64_t* const slot_all = reinterpret_cast<int64_t*>(cs_all + 2 * static_cast<size_t>(a.tokens_block) * a.rot);
  const int I = a.places;
  const int place = threadIdx.x % I, unit = threadIdx.x / I;
  const bool turned = place * 2 * V < a.rot;
  const int turns = half / V;   // places that are turned
  // This thread's 2V elements: V in the first half of the turned (or of the copied) elements and V in the second, so
  // that neighbouring threads' accesses are adjacent; an access of more than one element holds whole interleaved pairs.
  int p0 = place * V, p1 = half + place * V;
  if (V == 1 && a.interleaved) {
    p0 = 2 * place;
    p1 = p0 + 1;
  }
  if (!turned) {
    p0 = a.rot + (place - turns) * V;
    p1 = p0 + (a.d - a.rot) / 2;
  }
  const int n_units = kRopeThreads / I;

  const auto part_of = [&](int tile) {   // heads: queries, then keys, then values
    RopePart w;
    const uint32_t first = static_cast<uint32_t>(tile) * n_units, groups = a.groups;
    const uint32_t last = first + min(static_cast<uint32_t>(n_units), a.units - first) - 1;
    w.tok0 = static_cast<int>(first / groups);
    w.tok_n = static_cast<int>(last / groups) - w.tok0 + 1;
    const int tok = static_cast<int>((first + unit) / groups);
    const int group = static_cast<int>(first + unit - tok * groups);
    w.t = tok - w.tok0;
    w.kind = 0;
    w.head = group * U;
    int heads = a.H;
    if (kCache && group >= a.q_groups) {
      w.kind = group >= a.q_groups + a.kv_groups ? 2 : 1;
      w.head = (group - a.q_groups - (w.kind == 2 ? a.kv_groups : 0)) * U;
      heads = a.Hkv;
    }
    const bool idle = unit >= n_units || first + unit > last;
    w.n = idle || (w.kind == 0 && !turned && !a.tail) ? 0 : min(U, heads - w.head);
    return w;
  };
  const auto source = [&](const RopePart& w, int u) {
    const int64_t tok = w.tok0 + w.t;
    if (kCache && w.kind)
      return (w.kind == 1 ? static_cast<const TI*>(a.k) + tok * a.k_row : static_cast<const TI*>(a.v) + tok * a.v_row) +
             static_cast<int64_t>(w.head + u) * a.d;
    return static_cast<const TI*>(a.x) + tok * a.x_tok + (w.head + u) * a.x_head;
  };
  // A token's place in its sequence and the sequence; the page that the table has for it; the element offsets of K and V
  // there, or -1 for a token that is not written.
  const auto place_of = [&](int row) {
    return row < a.T ? make_int2(a.pos[row], a.seq ? a.seq[row] : row) : make_int2(-1, 0);
  };
  const auto page_of = [&](int2 at) {
    const int col = at.x < 0 ? 0 : at.x / a.page;
    if (at.x < 0 || at.y < 0 || at.y >= a.B || col >= a.table_cols) return -1;
    return a.table[static_cast<int64_t>(at.y) * a.table_stride + col];
  };
  const auto place_token = [&](int2 at, int id, int64_t* out) {
    int64_t ko = -1, vo = -1;
    if (at.x >= 0) {
      if (id >= 0 && id < a.n_pages) {
        const int in_page = at.x - at.x / a.page * a.page;
        ko = id * a.k_page + in_page * a.k_tok;
        vo = id * a.v_page + in_page * a.v_tok;
      } else if (a.status) {
        *a.status = HHR_ERR_BAD_INDEX;
      }
    }
    out[0] = ko;
    out[1] = vo;
  };
  const auto ask = [&](const RopePart& w, int buf) {   // each thread's own rows: no barrier between them and their use
    if constexpr (kStaged) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < w.n) {
          const TI* const src = source(w, u);
          const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(rows + ((buf * U + u) * 2) * kRopeThreads + threadIdx.x));
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src + p0) : "memory");
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + kRopeThreads * 16), "l"(src + p1) : "memory");
        }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };

  dependency_wait();
  launch_dependents();

  int tile = blockIdx.x, buf = 0;
  RopePart w = part_of(tile);
  ask(w, 0);
  Pack<TI, V> x0s[U], x1s[U];
  if constexpr (!kStaged) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < w.n) {
        load<TI, V>(source(w, u) + p0, x0s[u]);
        load<TI, V>(source(w, u) + p1, x1s[u]);
      }
  }
  // of this thread's token of the tile: its place and page; of the next tile's: its place
  int2 at = make_int2(-1, 0), at_next = at;
  int id = -1;
  const int duty = kRopeThreads - 1 - static_cast<int>(threadIdx.x);   // (the last warps have fewer angles to compute)
  const auto token_of = [&](const RopePart& part) { return duty < part.tok_n ? part.tok0 + duty : a.T; };
  if (kCache && duty < a.tokens_block) {
    at = place_of(token_of(w));
    if (kStaged && tile + gridDim.x < a.tiles) at_next = place_of(token_of(part_of(tile + gridDim.x)));
    id = page_of(at);
  }
  while (true) {
    const int next = kStaged ? tile + static_cast<int>(gridDim.x) : a.tiles;
    RopePart w_next = w;
    if (next < a.tiles) w_next = part_of(next);
    if (next >= a.tiles) w_next.n = 0;
    ask(w_next, buf ^ 1);

    // the angles of the tile's tokens, and their places in the cache, whose page was looked up while the tile before
    // was written
    float* const cs = cs_all + static_cast<size_t>(buf) * a.tokens_block * a.rot;
    int64_t* const slot = slot_all + static_cast<size_t>(buf) * a.tokens_block * 2;
    for (int i = threadIdx.x; i < w.tok_n * half; i += kRopeThreads) {
      const int ti = i / half, j = i - ti * half;
      const int p = (a.rope_pos ? a.rope_pos : a.pos)[w.tok0 + ti];
      const double turn = static_cast<double>(p) * a.freqs[j] * 0.15915494309189533577;
      const float r = static_cast<float>(2.0 * (turn - rint(turn)));
      float s, c;
      sincospif(r, &s, &c);
      int to = j / V, e = j % V;     // the place that pair j belongs to, and the which-th of its pairs
      if (V > 1 && a.interleaved) {
        const int access = 2 * j / V;
        to = access < turns ? access : access - turns;
        e = (2 * j - access * V) / 2 + (access < turns ? 0 : V / 2);
      }
      *reinterpret_cast<float2*>(cs + angle_at<V>(ti, half, turns, to, e)) =
          make_float2(a.mscale * c, a.sign * a.mscale * s);
    }
    if (kCache && duty < w.tok_n) place_token(at, id, slot + 2 * duty);
    // (one barrier a tile: the buffers of the tile after next are written behind the next one)
    __syncthreads();
    if constexpr (kStaged) asm volatile("cp.async.wait_group 1;" ::: "memory");

    int id_next = -1;
    int2 at_after = make_int2(-1, 0);
    if (kCache && duty < a.tokens_block && next < a.tiles) {
      id_next = page_of(at_next);
      if (next + gridDim.x < a.tiles) at_after = place_of(token_of(part_of(next + gridDim.x)));
    }

    const int n = kCache && w.n > 0 && slot[2 * w.t] < 0 ? 0 : w.n;
    const bool turn = turned && w.kind != 2;
    float cw[2 * V];       // cosines and sines of this place
    if (turn && n > 0) {
      if constexpr (V == 1) {
        const float2 z = *reinterpret_cast<const float2*>(cs + angle_at<V>(w.t, half, turns, place, 0));
        cw[0] = z.x;
        cw[1] = z.y;
      } else {
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const float4 z = *reinterpret_cast<const float4*>(cs + angle_at<V>(w.t, half, turns, place, e));
          cw[2 * e] = z.x;
          cw[2 * e + 1] = z.y;
          cw[2 * e + 2] = z.z;
          cw[2 * e + 3] = z.w;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u >= n) break;
      Pack<TI, V> x0, x1;
      if constexpr (kStaged) {
        x0 = rows[((buf * U + u) * 2) * kRopeThreads + threadIdx.x];
        x1 = rows[((buf * U + u) * 2 + 1) * kRopeThreads + threadIdx.x];
      } else {
        x0 = x0s[u];
        x1 = x1s[u];
      }
      const int64_t tok = w.tok0 + w.t;
      const bool is_q = !kCache || w.kind == 0;
      TI* const yq = static_cast<TI*>(a.y) + tok * a.y_tok + (w.head + u) * a.y_head;
      TC* yc = nullptr;
      if (!is_q)
        yc = w.kind == 2 ? static_cast<TC*>(a.V) + slot[2 * w.t + 1] + (w.head + u) * a.v_head
                         : static_cast<TC*>(a.K) + slot[2 * w.t] + (w.head + u) * a.k_head;
      if (!turn && (is_q || sizeof(TC) == sizeof(TI))) {   // the same type: the bits as they are
        TI* const y = is_q ? yq : reinterpret_cast<TI*>(yc);
        *reinterpret_cast<Pack<TI, V>*>(y + p0) = x0;
        *reinterpret_cast<Pack<TI, V>*>(y + p1) = x1;
        continue;
      }
      // halves: pair e is (f[e], f[V + e]); interleaved: (f[2e], f[2e + 1])
      float f[2 * V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        f[e] = to_f32(x0.v[e]);
        f[V + e] = to_f32(x1.v[e]);
      }
      if (turn) {
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float u1 = f[2 * e], u2 = f[2 * e + 1];
            f[2 * e] = fmaf(u1, cw[2 * e], -(u2 * cw[2 * e + 1]));
            f[2 * e + 1] = fmaf(u2, cw[2 * e], u1 * cw[2 * e + 1]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float u1 = f[e], u2 = f[V + e];
            f[e] = fmaf(u1, cw[2 * e], -(u2 * cw[2 * e + 1]));
            f[V + e] = fmaf(u2, cw[2 * e], u1 * cw[2 * e + 1]);
          }
        }
      }
      float f0[V], f1[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        f0[e] = f[e];
        f1[e] = f[V + e];
      }
      if (is_q) {
        store<TI, V>(yq + p0, f0, 1.0f);
        store<TI, V>(yq + p1, f1, 1.0f);
      } else {
        const float mul = w.kind == 2 ? a.v_inv : a.k_inv;
        store<TC, V>(yc + p0, f0, mul);
        store<TC, V>(yc + p1, f1, mul);
      }
    }
    if (next >= a.tiles) break;
    tile = next;
    w = w_next;
    buf ^= 1;
    at = at_next;
    id = id_next;
    at_next = at_after;
  }
}

// The accesses of a launch are 16 bytes wide where every row, and every place in a row, starts on 16 bytes (8 on the
// 8-bit side of an append); otherwise they go element by element.  Few tokens: a thread takes one head by plain loads, a
// block one tile (append of 256 tokens x 48 heads: 3.7 us, 5.4 staged).  Where four heads a thread still make four blocks an SM:
// three blocks an SM take the tiles in turn and stage the next one's rows in shared memory (8192 tokens, 40 heads of 128
// bf16: 58 us with one head a thread, 45 with two, 40 with four, 29 staged; two or four blocks an SM: 35, 33).
template <typename TI, typename TC, int V, bool kCache>
cudaError_t launch_rows(RopeArgs& a, cudaStream_t stream) {
  a.places = a.d / (2 * V);
  const int step = kRopeThreads / a.places;      // groups of a block
  const int64_t rows = static_cast<int64_t>(a.T) * (a.H + 2 * a.Hkv);
  int dev = 0, sms = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  if (cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) return e;
  const int U = a.H + 2 * a.Hkv >= 4 && rows >= static_cast<int64_t>(step) * 4 * (4 * sms) ? 4 : 1;
  a.q_groups = (a.H + U - 1) / U;
  a.kv_groups = (a.Hkv + U - 1) / U;
  a.groups = a.q_groups + 2 * a.kv_groups;
  a.units = static_cast<uint32_t>(a.T) * static_cast<uint32_t>(a.groups);
  a.tokens_block = std::min(step, (step - 2 + a.groups) / a.groups + 1);
  a.tiles = static_cast<int>((a.units - 1) / step + 1);
  const size_t smem = (V > 1 && U > 1 ? static_cast<size_t>(2 * U) * 2 * kRopeThreads * 16 : 0) +
                      2 * static_cast<size_t>(a.tokens_block) * (a.rot * sizeof(float) + 2 * sizeof(int64_t));
  static std::atomic<size_t> raised[2][kMaxDevices];
  const auto kern = U == 4 ? rope_kernel<TI, TC, V, 4, kCache> : rope_kernel<TI, TC, V, 1, kCache>;
  if (smem > 48 * 1024)
    if (cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), smem, raised[U == 4])) return e;
  const dim3 grid(static_cast<unsigned>(U == 4 && V > 1 ? std::min(a.tiles, sms * 3) : a.tiles));
  return launch_dependent<RopeArgs>(kern, grid, kRopeThreads, smem, stream, a);
}

template <typename TI, typename TC, bool kCache>
cudaError_t launch_typed(RopeArgs& a, bool wide, cudaStream_t stream) {
  return wide ? launch_rows<TI, TC, 16 / sizeof(TI), kCache>(a, stream) : launch_rows<TI, TC, 1, kCache>(a, stream);
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
    hi = std::min(std::ceil(dim(s->low)), rot - 1.0);   // (the published bound: beyond the last pair, which the ramp may not reach)
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
  a.H = H;
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
    case HHR_TYPE_BF16: return status_of(launch_typed<__nv_bfloat16, __nv_bfloat16, false>(a, wide, s));
    case HHR_TYPE_F16: return status_of(launch_typed<__half, __half, false>(a, wide, s));
    default: return status_of(launch_typed<float, float, false>(a, wide, s));
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
  const bool wide = a.rot % 16 == 0 && wide_row(k, k_row, 0, 2) && wide_row(v, v_row, 0, 2) &&
                    (!q || (wide_row(q, q_tok, 0, 2) && wide_row(q_out, q_out_tok, 0, 2)));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool e4m3 = c.kv_type == HHR_TYPE_E4M3;
  if (c.q_type == HHR_TYPE_BF16)
    return status_of(e4m3 ? launch_typed<__nv_bfloat16, __nv_fp8_e4m3, true>(a, wide, s)
                          : launch_typed<__nv_bfloat16, __nv_bfloat16, true>(a, wide, s));
  return status_of(e4m3 ? launch_typed<__half, __nv_fp8_e4m3, true>(a, wide, s) : launch_typed<__half, __half, true>(a, wide, s));
}

}  // extern "C"
