// The kernel of hhr_paged_attend: attention of one new token per sequence over
// a paged key-value cache, split over the cache's length and joined.
//
// out[h] = sum_n w_n V[n] / sum_n w_n with w_n = 2^(x_n - m), x_n = scale log2(e) q[h].K[n], m the largest x_n: one pass
// over K and V with a running m, rescaling what was summed whenever m grows; states of disjoint token ranges (m, sum w,
// sum w V) join by rescaling to the larger m.
//
// Bound: HBM.  A token costs 2 d elements of K and V per KV head and 4 d r operations for its r query heads: 2 to 24
// operations per byte, far below what the tensor cores do in that time, so the work is to keep loads in flight.
//
// Work.  A unit is (sequence, KV head, chunk of its query heads); its tokens are cut into tiles of 16.  The tiles of all
// units, one after another, are dealt out evenly: CTA c of G takes a contiguous range, so it ends one unit, does some
// whole ones and begins one, whatever the lengths are.  Lengths are read on the device (a captured call follows them);
// only a CTA's first and last unit are shared with its neighbours, so the exchanged states and counters take space for
// G CTAs and not for the sequences.  Of the CTAs that share a unit the last to arrive joins their states, in the CTAs'
// order: the result does not depend on which one that is.  No CTA waits for another.
//
// Tiles.  The CTA's warps take its tiles in turn.  Each warp copies its own tiles into its own ring (cp.async, 16 bytes
// a lane, swizzled) kDepth tiles ahead, across the borders of units, so no barrier stands between a load and its use
// and the loads go on while units are merged.  Rows are addressed one by one through the table, which takes any page
// size; where a page holds whole tiles one table entry serves all 16 rows.
//
// Products.  S^T = K Q^T (m16n8k16, tokens by heads: 8 heads fill n where a tile of 16 query rows would be half empty)
// and O^T += V^T P^T, float32 sums; P is the exact-to-2^-16 sum of two 16-bit values (2^-9 of P alone would show in a
// float32 output).  8-bit elements become fp16 in registers, exactly; bf16 queries of an 8-bit cache become fp16 after
// a power of two per row that makes their largest element about 2^14 (elements below 2^-28 of it lose bits).  mma.sync
// and not tcgen05: a tile is 16 tokens of one warp, whose P never leaves its registers; the tensor pipe has room to
// spare, and a 128-row tile with its commits would couple the warps that the private rings keep apart.
#pragma once

#include <algorithm>
#include <type_traits>

#include "hhr_internal.cuh"
#include "paged_common.cuh"

namespace hhr {

constexpr int kPagedMaxGrid = 160;   // CTAs that take part in a call (one per SM)

struct PagedArgs {
  const void* q;
  const void* K;
  const void* V;
  const int32_t* table;
  const int32_t* lens;
  void* out;
  float* lse;
  uint32_t* status;
  uint32_t* counters;          // [kPagedMaxGrid]: states that arrived for the unit a CTA began
  float* parts;                // [kPagedMaxGrid][2][part_stride]: states of a CTA's first and last unit
  int64_t q_seq, k_page, k_head, k_tok, v_page, v_head, v_tok;
  float scale_log2, v_scale;
  int B, Hq, Hkv, page, n_pages, table_cols, table_stride, window, out_f32;
  int r, chunk, chunks;        // query heads of a KV head, of a unit (at most 8 NT), and units of a KV head
  int part_stride;             // floats
  uint32_t page_magic;         // n / page = (umulhi(n, magic) + n) >> shift for n < 2^31
  int page_shift;
  int min_tiles;               // a CTA takes at least that many
};

// Floats of an exchanged state: [heads][d] sums, [heads][2] maximum and weight sum.
inline int paged_part_stride(int heads, int d) { return (heads * (d + 2) + 3) / 4 * 4; }

template <typename TQ, typename TC, int D, int NT>
struct PagedShape {
  using TM = std::conditional_t<std::is_same<TC, __nv_bfloat16>::value, __nv_bfloat16, __half>;   // of the products
  static constexpr bool kE4 = sizeof(TC) == 1;
  static constexpr int kRow = D * static_cast<int>(sizeof(TC));   // bytes of a row
  static constexpr int kTile = 16 * kRow;
  static constexpr int kWarps = kRow > 256 ? 4 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kDepth = std::min(8, 196608 / (kWarps * 2 * kTile));
  static constexpr int kMergeD = std::min(D, 128);                // columns of a merge pass, of 4 heads
  static constexpr int kMergeStride = kMergeD + 4;
  static constexpr int kHeads = 8 * NT;
  // registers hold the query fragments where they are few, otherwise every tile reads them from shared memory
  static constexpr bool kQRegs = D / 16 * NT * 2 <= 32;
  // shared memory
  static constexpr int kRing = 0;
  static constexpr int kMerge = kRing + kWarps * kDepth * 2 * kTile;
  // a merge pass of all warps; the weights of 8 heads, their inverse sums and the threads' sums of a join
  static constexpr int kMergeFloats = std::max(kWarps * 4 * kMergeStride, 8 * kPagedMaxGrid + 8 + 4 * kThreads);
  static constexpr int kMl = kMerge + kMergeFloats * 4;
  static constexpr int kQ = kMl + kWarps * kHeads * 8;
  static constexpr int kQs = kQ + kHeads * D * 2;
  static constexpr int kMasks = kQs + kHeads * 4;
  static constexpr int kSmem = kMasks + kWarps * kDepth * 4;
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};

// Tiles of a sequence: [first, end).
struct TileRange {
  int lo, len, first, end;
};

__device__ __forceinline__ TileRange tile_range(const PagedArgs& a, int b) {
  TileRange t;
  t.len = a.lens[b];
  if (t.len < 0 || t.len > a.table_cols * a.page) t.len = 0;
  t.lo = a.window ? max(0, t.len - a.window) : 0;
  t.first = t.lo >> 4;
  t.end = (t.len + 15) >> 4;
  return t;
}

__device__ __forceinline__ int page_of(const PagedArgs& a, int n) {
  return static_cast<int>((__umulhi(static_cast<uint32_t>(n), a.page_magic) + static_cast<uint32_t>(n)) >> a.page_shift);
}

// A tile of the call: sequence, unit of the sequence, tile of the unit.
struct TileCursor {
  TileRange t;
  int b, u, at;
  __device__ __forceinline__ void advance(const PagedArgs& a, int units, int by) {   // the target has to exist
    at += by;
    while (at >= t.end) {
      const int over = at - t.end;
      if (++u == units) {
        u = 0;
        do t = tile_range(a, ++b);
        while (t.first >= t.end);
      }
      at = t.first + over;
    }
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <typename TM>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<TM, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two floats as a pair of 16-bit values (hi) and what they leave (lo).
template <typename TM>
__device__ __forceinline__ void split(float x, float y, uint32_t& hi, uint32_t& lo) {
  if constexpr (std::is_same<TM, __half>::value) {
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    const float2 f = __bfloat1622float2(h);
    const __nv_bfloat162 l = __floats2bfloat162_rn(x - f.x, y - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
  }
}

// The two e4m3 values of the low (high) half of x as fp16, exactly.
__device__ __forceinline__ uint32_t wide_lo(uint32_t x) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(x & 0xffffu), __NV_E4M3);
  return static_cast<uint32_t>(h.x) | (static_cast<uint32_t>(h.y) << 16);
}
__device__ __forceinline__ uint32_t wide_hi(uint32_t x) { return wide_lo(x >> 16); }

// Byte offset of 16-byte chunk c of row i in a tile of rows of `row` bytes: eight rows read at the same chunk, or one
// row's chunks, fall on different banks.
template <int row>
__device__ __forceinline__ int swizzled(int i, int c) {
  return i * row + ((c ^ (row >= 128 ? (i & 7) : ((i >> 1) & 3))) << 4);
}

template <typename TQ, typename TC, int D, int NT>
__global__ void __launch_bounds__(PagedShape<TQ, TC, D, NT>::kThreads, 1) paged_kernel(const PagedArgs a) {
  using S = PagedShape<TQ, TC, D, NT>;
  using TM = typename S::TM;
  constexpr int kWarps = S::kWarps, kThreads = S::kThreads, kDepth = S::kDepth, kRow = S::kRow, kTile = S::kTile;
  constexpr int kLead = 2 * kDepth - 1;    // copy groups that may be in flight behind the one that is waited for
  constexpr float kLift = std::is_same<TM, __half>::value ? 14.0f : 0.0f;   // weights up to 2^14: fp16 keeps 2^-38 of the largest
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int64_t s_scan[kWarps];
  __shared__ int64_t s_pre;
  __shared__ int s_b, s_last;
  float* const s_merge = reinterpret_cast<float*>(smem + S::kMerge);
  float2* const s_ml = reinterpret_cast<float2*>(smem + S::kMl);
  float* const s_qs = reinterpret_cast<float*>(smem + S::kQs);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int units = a.Hkv * a.chunks;

  dependency_wait();
  launch_dependents();

  // Rows of sequences without tokens, and lengths out of range.
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    const int len = a.lens[b];
    if (len < 0 || len > a.table_cols * a.page) {
      if (tid == 0) *a.status = HHR_ERR_BAD_INDEX;
    } else if (len > 0) {
      continue;
    }
    const size_t row = static_cast<size_t>(b) * a.Hq;
    for (int e = tid; e < a.Hq * D; e += kThreads) {
      if (a.out_f32)
        static_cast<float*>(a.out)[row * D + e] = 0.0f;
      else
        static_cast<TQ*>(a.out)[row * D + e] = from_f32<TQ>(0.0f);
    }
    if (a.lse)
      for (int h = tid; h < a.Hq; h += kThreads) a.lse[row + h] = -INFINITY;
  }

  // This CTA's range [f0, f1) of the tiles of all units; thread i sums the tiles of its run of sequences.
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b_lo = min(tid * per, a.B), b_hi = min(b_lo + per, a.B);
  int64_t mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const TileRange t = tile_range(a, b);
    mine += max(0, t.end - t.first);
  }
  int64_t upto = mine;
#pragma unroll
  for (int w = 1; w < 32; w <<= 1) {
    const int64_t x = __shfl_up_sync(~0u, upto, w);
    if (lane >= w) upto += x;
  }
  if (lane == 31) s_scan[warp] = upto;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) upto += s_scan[w];
    total += s_scan[w];
  }
  total *= units;
  const int G = static_cast<int>(min(static_cast<int64_t>(gridDim.x), max(int64_t{1}, total / a.min_tiles)));
  const int c = blockIdx.x;
  if (total == 0 || c >= G) return;
  const int64_t quot = total / G, rem = total % G;
  const int64_t f0 = quot * c + min(static_cast<int64_t>(c), rem), f1 = f0 + quot + (c < rem ? 1 : 0);
  const int64_t before = (upto - mine) * units;
  if (before <= f0 && f0 < upto * units) {
    int64_t pre = upto - mine;
    int b = b_lo;
    for (;; ++b) {
      const TileRange t = tile_range(a, b);
      const int n = max(0, t.end - t.first);
      if (f0 < (pre + n) * units) break;
      pre += n;
    }
    s_b = b;
    s_pre = pre;
  }
  __syncthreads();
  TileCursor seg;    // the unit being attended
  seg.b = s_b;
  seg.t = tile_range(a, seg.b);
  {
    const int64_t off = f0 - s_pre * units;
    const int n = seg.t.end - seg.t.first;
    seg.u = static_cast<int>(off / n);
    seg.at = seg.t.first + static_cast<int>(off - static_cast<int64_t>(seg.u) * n);
  }

  // ---- loads: this warp's tiles f0 + warp, f0 + warp + kWarps, ...
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem + S::kRing)) + warp * kDepth * 2 * kTile;
  uint32_t* const masks = reinterpret_cast<uint32_t*>(smem + S::kMasks) + warp * kDepth;
  constexpr int kChunks = kRow / 16;               // 16-byte chunks of a row
  constexpr int kCopies = kChunks / 2;             // copies of a lane per 16 rows
  constexpr int kRowStep = kChunks >= 32 ? 1 : 32 / kChunks;   // rows of a warp's copy
  const int row0 = lane / kChunks, chunk0 = lane % kChunks;
  const bool whole = (a.page & 15) == 0;           // tiles do not cross pages
  const unsigned char* const Kb = static_cast<const unsigned char*>(a.K);
  const unsigned char* const Vb = static_cast<const unsigned char*>(a.V);
  TileCursor ld = seg;
  int64_t ld_f = f0 + warp;
  const unsigned char *Kh = Kb, *Vh = Vb;   // of the tile's KV head
  int id = 0, in_page = 0;     // of row lane & 15 (of the tile's first row, if whole)
  uint32_t mask = 0;           // the tile's rows that are tokens
  const auto find = [&]() {    // the page of the tile at ld
    const int n0 = ld.at * 16, n = whole ? n0 : n0 + (lane & 15);
    const int row = n0 + (lane & 15);
    const bool in = row >= ld.t.lo && row < ld.t.len;
    const int p = page_of(a, n);
    in_page = n - p * a.page;
    id = 0;
    if (whole || in) id = a.table[static_cast<int64_t>(ld.b) * a.table_stride + p];
    mask = __ballot_sync(~0u, in) & 0xffffu;
    const int kv = a.chunks == 1 ? ld.u : ld.u / a.chunks;
    Kh = Kb + kv * a.k_head * static_cast<int>(sizeof(TC));
    Vh = Vb + kv * a.v_head * static_cast<int>(sizeof(TC));
  };
  uint32_t live = 0;           // its rows that are copied
  int live_id = 0;
  const auto copy_rows = [&](uint32_t dst, const unsigned char* base, int64_t page, int64_t tok) {
    if (whole) {
      const unsigned char* src = base + (live_id * page + (in_page + row0) * tok) * static_cast<int>(sizeof(TC)) + chunk0 * 16;
      const int64_t step = tok * (kRowStep * static_cast<int>(sizeof(TC)));
#pragma unroll
      for (int j = 0; j < kCopies; ++j) {
        const int row = j * kRowStep + row0;
        copy16(dst + swizzled<kRow>(row, chunk0), src, (live >> row) & 1);
        src += step;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kCopies; ++j) {
        const int row = j * kRowStep + row0;
        const int64_t rid = __shfl_sync(~0u, live_id, row), rin = __shfl_sync(~0u, in_page, row);
        const bool on = (live >> row) & 1;
        const unsigned char* src = base + (rid * page + rin * tok) * static_cast<int>(sizeof(TC)) + chunk0 * 16;
        copy16(dst + swizzled<kRow>(row, chunk0), on ? src : base, on);
      }
    }
  };
  // K, then V, of the tile at ld go to a slot; the two calls of a tile stand around the next tile's products
  const auto issue_k = [&](int slot) {
    if (ld_f < f1) {
      const bool ok = static_cast<uint32_t>(id) < static_cast<uint32_t>(a.n_pages);
      if (whole) {
        live = ok ? mask : 0;
      } else {
        live = mask & __ballot_sync(~0u, ok);
      }
      live_id = ok ? id : 0;
      if (lane == 0) {
        masks[slot] = live;
        if (live != mask) *a.status = HHR_ERR_BAD_INDEX;
      }
      copy_rows(ring + slot * 2 * kTile, Kh, a.k_page, a.k_tok);
    }
    copy_commit();
  };
  const auto issue_v = [&](int slot) {
    if (ld_f < f1) {
      copy_rows(ring + slot * 2 * kTile + kTile, Vh, a.v_page, a.v_tok);
      ld_f += kWarps;
      if (ld_f < f1) {
        ld.advance(a, units, kWarps);
        find();
      }
    }
    copy_commit();
  };
  if (ld_f < f1) {
    if (warp) ld.advance(a, units, warp);
    find();
  }
#pragma unroll
  for (int s = 0; s < kDepth; ++s) {
    issue_k(s);
    issue_v(s);
  }

  const uint32_t q_smem = static_cast<uint32_t>(__cvta_generic_to_shared(smem + S::kQ));
  int slot = 0;
  int64_t f = f0 + warp, seg_f = f0;

  while (true) {   // units of this CTA's range
    const int g_kv = seg.u / a.chunks, first_head = (seg.u - g_kv * a.chunks) * a.chunk;
    const int heads = min(a.chunk, a.r - first_head);
    const int head0 = g_kv * a.r + first_head;
    const int64_t unit_f0 = seg_f - (seg.at - seg.t.first);
    const int64_t unit_f1 = unit_f0 + (seg.t.end - seg.t.first);
    const int64_t seg_f1 = min(f1, unit_f1);

    // queries: a warp per head
    for (int h = warp; h < S::kHeads; h += kWarps) {
      constexpr int E = D / 32;
      float x[E];
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = 0;
      if (h < heads) {
        const Pack<TQ, E> v = *reinterpret_cast<const Pack<TQ, E>*>(
            static_cast<const TQ*>(a.q) + seg.b * a.q_seq + static_cast<int64_t>(head0 + h) * D + lane * E);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = to_f32(v.v[e]);
      }
      float sc = a.scale_log2;
      if constexpr (std::is_same<TQ, __nv_bfloat16>::value && std::is_same<TM, __half>::value) {
        float top = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) top = fmaxf(top, fabsf(x[e]));
#pragma unroll
        for (int w = 16; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, w));
        const int up = top > 0 && top < INFINITY ? 14 - ilogbf(top) : 0;
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = ldexpf(x[e], up);
        sc = ldexpf(sc, -up);
      }
      if (lane == 0) s_qs[h] = sc;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const int at = lane * E + e;     // 8-bit keys: the order in which their 4-byte groups fill a fragment
        const int to = S::kE4 ? (at & ~15) + ((at & 2) ? 8 : 0) + ((at & 12) >> 1) : at;
        Pack<TM, 2> y;
        y.v[0] = from_f32<TM>(x[e]);
        y.v[1] = from_f32<TM>(x[e + 1]);
        *reinterpret_cast<Pack<TM, 2>*>(smem + S::kQ + swizzled<2 * D>(h, to >> 3) + (to & 7) * 2) = y;
      }
    }
    __syncthreads();
    uint32_t qf[S::kQRegs ? D / 16 : 1][NT][2];
    const auto q_frag = [&](int kk, uint32_t (&b)[NT][2]) {
#pragma unroll
      for (int n = 0; n < NT; n += 2) {
        uint32_t r[4];
        const int row = n * 8 + (lane & 7) + (n + 1 < NT ? (lane >> 4) * 8 : 0);
        ldsm4(r, q_smem + swizzled<2 * D>(row, kk * 2 + ((lane >> 3) & 1)));
        b[n][0] = r[0];
        b[n][1] = r[1];
        if (n + 1 < NT) {
          b[n + 1][0] = r[2];
          b[n + 1][1] = r[3];
        }
      }
    };
    if constexpr (S::kQRegs)
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) q_frag(kk, qf[kk]);
    float sc[NT][2], m[NT][2], base[NT][2], l[NT][2], o[NT][D / 16][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sc[n][e] = s_qs[n * 8 + 2 * t4 + e];
        m[n][e] = -INFINITY;
        base[n][e] = l[n][e] = 0;
      }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][j][e] = 0;

    for (; f < seg_f1; f += kWarps) {
      const uint32_t kt = ring + slot * 2 * kTile, vt = kt + kTile;
      copy_wait<kLead>();
      __syncwarp();
      const uint32_t rows = masks[slot];
      // S^T = K Q^T, even and odd steps in sums of their own
      float s[2][NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[0][n][e] = s[1][n][e] = 0;
      const auto dot = [&](int kk, const uint32_t (&r)[4]) {
        uint32_t bq[NT][2];
        if constexpr (S::kQRegs) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            bq[n][0] = qf[kk][n][0];
            bq[n][1] = qf[kk][n][1];
          }
        } else {
          q_frag(kk, bq);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) mma<TM>(s[kk & 1][n], r, bq[n][0], bq[n][1]);
      };
#pragma unroll
      for (int kk = 0; kk < D / 16; kk += S::kE4 ? 2 : 1) {
        uint32_t r[4];
        ldsm4(r, kt + swizzled<kRow>(lane & 15, (S::kE4 ? kk : 2 * kk) + (lane >> 4)));
        if constexpr (S::kE4) {
          // a lane's 4 bytes fill two of the fragment's places: the order of the queries' elements follows that
          dot(kk, {wide_lo(r[0]), wide_lo(r[1]), wide_hi(r[0]), wide_hi(r[1])});
          dot(kk + 1, {wide_lo(r[2]), wide_lo(r[3]), wide_hi(r[2]), wide_hi(r[3])});
        } else {
          dot(kk, r);
        }
      }
      __syncwarp();
      issue_k(slot);
      // weights: lane (g, t4) holds tokens g and g + 8 of heads 2 t4 and 2 t4 + 1
      bool grown = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[0][n][e] = (s[0][n][e] + s[1][n][e]) * sc[n][e & 1];
        if (rows != 0xffffu) {
          if (!((rows >> g) & 1)) s[0][n][0] = s[0][n][1] = -INFINITY;
          if (!((rows >> (g + 8)) & 1)) s[0][n][2] = s[0][n][3] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) grown = grown || fmaxf(s[0][n][e], s[0][n][e + 2]) > m[n][e];
      }
      if (__any_sync(~0u, grown)) {   // rare after the first tiles
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(m[n][e], fmaxf(s[0][n][e], s[0][n][e + 2]));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 4));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 16));
            const float by = top == m[n][e] ? 1.0f : ex2(m[n][e] - top);
            m[n][e] = top;
            base[n][e] = top == -INFINITY ? 0.0f : top - kLift;
            l[n][e] *= by;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              o[n][j][e] *= by;
              o[n][j][e + 2] *= by;
            }
          }
      }
      uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = ex2(s[0][n][e] - base[n][e & 1]);
        l[n][0] += w[0] + w[2];
        l[n][1] += w[1] + w[3];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          split<TM>(w[2 * e], w[2 * e + 1], hi[n][e], lo[n][e]);
          hi[n][e] = transposed(hi[n][e]);
          lo[n][e] = transposed(lo[n][e]);
        }
      }
      copy_wait<kLead>();
      __syncwarp();
      // O^T += V^T P^T
      const auto add = [&](int j, const uint32_t (&r)[4]) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma<TM>(o[n][j], r, hi[n][0], hi[n][1]);
          mma<TM>(o[n][j], r, lo[n][0], lo[n][1]);
        }
      };
#pragma unroll
      for (int j = 0; j < D / 16; j += S::kE4 ? 2 : 1) {
        uint32_t r[4];
        if constexpr (S::kE4) {
          // a transposed 2-byte element is columns 2 g and 2 g + 1 of a token: rows g and g + 8 of the product
          ldsm4_trans(r, vt + swizzled<kRow>(lane & 15, j + (lane >> 4)));
#pragma unroll
          for (int e = 0; e < 4; ++e) r[e] = __byte_perm(r[e], 0, 0x3120);
          add(j, {wide_lo(r[0]), wide_hi(r[0]), wide_lo(r[1]), wide_hi(r[1])});
          add(j + 1, {wide_lo(r[2]), wide_hi(r[2]), wide_lo(r[3]), wide_hi(r[3])});
        } else {
          ldsm4_trans(r, vt + swizzled<kRow>((lane & 7) + (lane >> 4) * 8, 2 * j + ((lane >> 3) & 1)));
          add(j, r);
        }
      }
      __syncwarp();
      issue_v(slot);
      slot = slot + 1 == kDepth ? 0 : slot + 1;
    }

    // ---- the warps' states of this unit, joined
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[n][e] += __shfl_xor_sync(~0u, l[n][e], w);
        if (g == 0)
          s_ml[warp * S::kHeads + n * 8 + 2 * t4 + e] = make_float2(m[n][e] == -INFINITY ? -INFINITY : base[n][e], l[n][e]);
      }
    const bool whole_unit = seg_f == unit_f0 && seg_f1 == unit_f1;
    const auto owner = [&](int64_t x) {
      const int64_t wide = rem * (quot + 1);
      return static_cast<int>(x < wide ? x / (quot + 1) : rem + (x - wide) / quot);
    };
    const int c0 = whole_unit ? c : owner(unit_f0);
    float* const part = a.parts + static_cast<size_t>(2 * c + (c == c0)) * a.part_stride;
    const size_t out_row = static_cast<size_t>(seg.b) * a.Hq + head0;
    const auto finish = [&](int h, int d, float y) {
      const size_t at = (out_row + h) * D + d;
      if (a.out_f32)
        static_cast<float*>(a.out)[at] = y;
      else
        static_cast<TQ*>(a.out)[at] = from_f32<TQ>(y);
    };
    const auto weight = [](float m, float top) { return m == top ? 1.0f : ex2(m - top); };
    const auto inverse = [&](float sum) { return sum > 0 ? a.v_scale / sum : sum; };   // 0 for none, NaN stays
    const auto log_sum = [](float top, float sum) { return sum == 0 ? -INFINITY : (top + log2f(sum)) * 0.69314718055994530942f; };
#pragma unroll
    for (int h4 = 0; h4 < 2 * NT; ++h4)
#pragma unroll
      for (int d0 = 0; d0 < D; d0 += S::kMergeD) {
        const int n_heads = min(4, heads - 4 * h4);
        if (n_heads <= 0) break;
        if ((t4 >> 1) == (h4 & 1)) {
          float* const to = s_merge + (warp * 4 + 2 * (t4 & 1)) * S::kMergeStride;
#pragma unroll
          for (int j = 0; j < S::kMergeD / 16; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float y0 = o[h4 / 2][d0 / 16 + j][e], y1 = o[h4 / 2][d0 / 16 + j][e + 2];
              float* const at = to + e * S::kMergeStride + j * 16;
              if constexpr (S::kE4) {
                *reinterpret_cast<float2*>(at + 2 * g) = make_float2(y0, y1);
              } else {
                at[g] = y0;
                at[g + 8] = y1;
              }
            }
        }
        __syncthreads();
        for (int e = tid * 2; e < n_heads * S::kMergeD; e += kThreads * 2) {
          const int h = e / S::kMergeD, d = e % S::kMergeD;
          const float2* const ml = s_ml + 4 * h4 + h;
          float top = -INFINITY, sum = 0;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w * S::kHeads].x);
          float2 y = make_float2(0, 0);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 s = ml[w * S::kHeads];
            const float by = weight(s.x, top);
            const float2 x = *reinterpret_cast<const float2*>(s_merge + (w * 4 + h) * S::kMergeStride + d);
            sum = fmaf(s.y, by, sum);
            y.x = fmaf(x.x, by, y.x);
            y.y = fmaf(x.y, by, y.y);
          }
          const int head = 4 * h4 + h;
          if (whole_unit) {
            const float inv = inverse(sum);
            finish(head, d0 + d, y.x * inv);
            finish(head, d0 + d + 1, y.y * inv);
            if (d0 + d == 0 && a.lse) a.lse[out_row + head] = log_sum(top, sum);
          } else {
            *reinterpret_cast<float2*>(part + head * D + d0 + d) = y;
            if (d0 + d == 0) *reinterpret_cast<float2*>(part + heads * D + 2 * head) = make_float2(top, sum);
          }
        }
        __syncthreads();
      }

    if (!whole_unit) {
      // The last of the unit's CTAs to arrive joins their states from L2.
      const int n_parts = owner(unit_f1 - 1) - c0 + 1;
      if (tid == 0) {
        __threadfence();
        const bool last = atomicAdd(a.counters + c0, 1u) == static_cast<uint32_t>(n_parts - 1);
        if (last) a.counters[c0] = 0;
        __threadfence();
        s_last = last;
      }
      __syncthreads();
      if (s_last) {
        float* const by = s_merge;                             // [8][n_parts]
        float* const invs = s_merge + 8 * kPagedMaxGrid;       // [8]
        float4* const sums = reinterpret_cast<float4*>(invs + 8);   // [kThreads]
        const auto part_of = [&](int i) {
          return a.parts + static_cast<size_t>(2 * (c0 + i) + (i == 0)) * a.part_stride;
        };
        for (int h0 = 0; h0 < heads; h0 += 8) {
          const int n_heads = min(8, heads - h0);
          for (int h = warp; h < n_heads; h += kWarps) {
            float top = -INFINITY, sum = 0;
            for (int i = lane; i < n_parts; i += 32)
              top = fmaxf(top, __ldcg(part_of(i) + heads * D + 2 * (h0 + h)));
#pragma unroll
            for (int w = 16; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, w));
            for (int i = lane; i < n_parts; i += 32) {
              const float2 s = __ldcg(reinterpret_cast<const float2*>(part_of(i) + heads * D + 2 * (h0 + h)));
              const float x = weight(s.x, top);
              by[h * n_parts + i] = x;
              sum = fmaf(s.y, x, sum);
            }
#pragma unroll
            for (int w = 16; w; w >>= 1) sum += __shfl_xor_sync(~0u, sum, w);
            if (lane == 0) {
              invs[h] = inverse(sum);
              if (a.lse) a.lse[out_row + h0 + h] = log_sum(top, sum);
            }
          }
          __syncthreads();
          const int items = n_heads * (D / 4);                 // 4 columns each
          const int splits = max(1, kThreads / items);         // parts are dealt out where there are few items
          for (int e0 = 0; e0 < items; e0 += kThreads) {
            const int e = splits > 1 ? tid % items : e0 + tid, sp = splits > 1 ? tid / items : 0;
            float4 y = make_float4(0, 0, 0, 0);
            if (e < items && sp < splits) {
              const int h = e / (D / 4);
#pragma unroll 8
              for (int i = sp; i < n_parts; i += splits) {
                const float4 x = __ldcg(reinterpret_cast<const float4*>(part_of(i) + h0 * D) + e);
                const float k = by[h * n_parts + i];
                y.x = fmaf(x.x, k, y.x);
                y.y = fmaf(x.y, k, y.y);
                y.z = fmaf(x.z, k, y.z);
                y.w = fmaf(x.w, k, y.w);
              }
            }
            if (splits > 1) {
              sums[tid] = y;
              __syncthreads();
              if (tid < items)
                for (int i = 1; i < splits; ++i) {
                  const float4 x = sums[i * items + tid];
                  y.x += x.x;
                  y.y += x.y;
                  y.z += x.z;
                  y.w += x.w;
                }
            }
            if (e < items && sp == 0) {
              const int h = e / (D / 4), d = e % (D / 4) * 4;
              const float inv = invs[h];
              finish(h0 + h, d, y.x * inv);
              finish(h0 + h, d + 1, y.y * inv);
              finish(h0 + h, d + 2, y.z * inv);
              finish(h0 + h, d + 3, y.w * inv);
            }
          }
          __syncthreads();
        }
      }
    }
    seg_f = seg_f1;
    if (seg_f >= f1) break;
    seg.at = seg.t.end - 1;
    seg.advance(a, units, 1);
  }
}

// Launches the variant for D and the heads of a unit.
template <typename TQ, typename TC, int D, int NT>
cudaError_t launch_paged_kernel(const PagedArgs& a, int grid, cudaStream_t s) {
  using S = PagedShape<TQ, TC, D, NT>;
  static std::atomic<size_t> raised[kMaxDevices];
  const auto kern = paged_kernel<TQ, TC, D, NT>;
  if (cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), S::kSmem, raised)) return e;
  return launch_dependent<PagedArgs>(kern, dim3(grid), S::kThreads, S::kSmem, s, a);
}

// Most heads of a unit, by the registers of its sums: D / 16 x 4 floats a lane for 8 heads.
inline int paged_max_heads(int d) { return d == 64 ? 32 : d == 128 ? 24 : 16; }

template <typename TQ, typename TC>
cudaError_t launch_paged_typed(const PagedArgs& a, int d, int grid, cudaStream_t s) {
  const int nt = (a.chunk + 7) / 8;
  if (d == 64) {
    if (nt == 1) return launch_paged_kernel<TQ, TC, 64, 1>(a, grid, s);
    if (nt == 2) return launch_paged_kernel<TQ, TC, 64, 2>(a, grid, s);
    if (nt == 3) return launch_paged_kernel<TQ, TC, 64, 3>(a, grid, s);
    return launch_paged_kernel<TQ, TC, 64, 4>(a, grid, s);
  }
  if (d == 128) {
    if (nt == 1) return launch_paged_kernel<TQ, TC, 128, 1>(a, grid, s);
    if (nt == 2) return launch_paged_kernel<TQ, TC, 128, 2>(a, grid, s);
    return launch_paged_kernel<TQ, TC, 128, 3>(a, grid, s);
  }
  if (nt == 1) return launch_paged_kernel<TQ, TC, 256, 1>(a, grid, s);
  return launch_paged_kernel<TQ, TC, 256, 2>(a, grid, s);
}

// One translation unit per pair of types (paged_*.cu).
cudaError_t launch_paged_bf16(const PagedArgs& a, int d, int grid, cudaStream_t s);
cudaError_t launch_paged_f16(const PagedArgs& a, int d, int grid, cudaStream_t s);
cudaError_t launch_paged_bf16_e4m3(const PagedArgs& a, int d, int grid, cudaStream_t s);
cudaError_t launch_paged_f16_e4m3(const PagedArgs& a, int d, int grid, cudaStream_t s);

}  // namespace hhr
