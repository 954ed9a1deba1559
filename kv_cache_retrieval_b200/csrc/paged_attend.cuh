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
// Work.  A unit is (sequence, KV head, chunk of its query heads); its tokens are cut into tiles of 16 or 32.  The tiles
// of all units, one after another, are dealt out evenly: every warp of the card takes a contiguous range, so it ends one
// unit, does some whole ones and begins one, whatever the lengths are.  Lengths are read on the device (a captured call
// follows them).  A whole unit is written by its warp alone; the states of a unit that several warps share are joined by
// their CTA when its warps are done, and by the last of its CTAs to arrive if it has several: always in the order of
// the tokens, so the result does not depend on which one that is.  Only a CTA's first and last unit are shared with its
// neighbours: the workspace is for the card's CTAs and not for the sequences.  No CTA waits for another.
//
// Tiles.  Each warp copies its tiles into its own ring (cp.async, 16 bytes a lane, swizzled) kDepth tiles ahead, across
// the borders of units: no barrier stands anywhere before the join, and loads go on while a unit ends.  Rows are
// addressed one by one through the table, which takes any page size; where a page holds whole 16-row tiles one table
// entry serves all of them.
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
  float* parts;                // [kPagedMaxGrid][2]: joined states of a CTA's first and last unit
  float* firsts;               // [kPagedMaxGrid][8]: states of the units that a warp ends and did not begin
  int64_t q_seq, k_page, k_head, k_tok, v_page, v_head, v_tok;
  float scale_log2, v_scale;
  int B, Hq, Hkv, page, n_pages, table_cols, table_stride, window, out_f32;
  int r, chunk, chunks;        // query heads of a KV head, of a unit (at most 8 NT), and units of a KV head
  int state;                   // floats of a state
  uint32_t page_magic;         // n / page = (umulhi(n, magic) + n) >> shift for n < 2^31
  int page_shift;
  int min_tiles;               // a warp takes at least that many
};

// Floats of a state: a row of d sums of each head, then its maximum and weight sum (rows of d + 4 floats fall on
// different banks).
inline int paged_state(int heads, int d) { return heads * (d + 4); }

template <typename TQ, typename TC, int D, int NT>
struct PagedShape {
  using TM = std::conditional_t<std::is_same<TC, __nv_bfloat16>::value, __nv_bfloat16, __half>;   // of the products
  static constexpr bool kE4 = sizeof(TC) == 1;
  static constexpr int kRow = D * static_cast<int>(sizeof(TC));   // bytes of a row
  static constexpr int kSub = kRow <= 128 ? 2 : 1;                // 16-row products of a tile
  static constexpr int kTokens = 16 * kSub;
  static constexpr int kTile = kTokens * kRow;
  static constexpr int kHeads = 8 * NT;
  // registers hold the query fragments unless the sums leave no room: then each warp reads them from shared memory
  static constexpr bool kQRegs = D / 16 * NT * 2 <= 48;
  static constexpr int kWarps = kRow > 256 || !kQRegs ? 4 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kDepth = std::min(8, 196608 / (kWarps * 2 * kTile));
  // shared memory
  static constexpr int kRing = 0;
  static constexpr int kRingWarp = kDepth * 2 * kTile;            // of a warp; in the end it holds the warp's last state
  static constexpr int kQ = kRing + kWarps * kRingWarp;
  static constexpr int kQWarp = kQRegs ? 0 : kHeads * D * 2;
  // the join: weights of 8 heads, their inverse sums, the threads' sums
  static constexpr int kJoin = (8 * kPagedMaxGrid + 8 + 4 * kThreads) * 4;
  static constexpr int kMasks = kQ + std::max(kWarps * kQWarp, kJoin);
  static constexpr int kSmem = kMasks + kWarps * kDepth * 4;
  static_assert(kSmem <= 226 * 1024, "shared memory of a CTA");
  static_assert(kHeads * (D + 4) * 4 <= kRingWarp, "a warp's state lies in its ring");
};

// Tiles of a sequence: [first, end).
struct TileRange {
  int lo, len, first, end;
};

template <int kTokens>
__device__ __forceinline__ TileRange tile_range(const PagedArgs& a, int b) {
  TileRange t;
  t.len = a.lens[b];
  if (t.len < 0 || t.len > a.table_cols * a.page) t.len = 0;
  t.lo = a.window ? max(0, t.len - a.window) : 0;
  t.first = t.lo / kTokens;
  t.end = static_cast<int>((static_cast<uint32_t>(t.len) + (kTokens - 1)) / kTokens);
  return t;
}

__device__ __forceinline__ int page_of(const PagedArgs& a, int n) {
  return static_cast<int>((__umulhi(static_cast<uint32_t>(n), a.page_magic) + static_cast<uint32_t>(n)) >> a.page_shift);
}

// A tile of the call: sequence, unit of the sequence, tile of the unit.
struct TileCursor {
  TileRange t;
  int b, u, at;
  template <int kTokens>
  __device__ __forceinline__ void next(const PagedArgs& a, int units) {   // the next tile has to exist
    if (++at < t.end) return;
    if (++u == units) {
      u = 0;
      do t = tile_range<kTokens>(a, ++b);
      while (t.first >= t.end);
    }
    at = t.first;
  }
};

// An open state: one of several of its unit.
struct OpenState {
  int64_t x0, x1;       // the unit's tiles
  const float* at;
  int b, u;
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

// The weight of a state of maximum m among states of maximum top; 1 / sum of a unit's weights (0 for none, NaN stays)
// and its log-sum-exp.
__device__ __forceinline__ float paged_weight(float m, float top) { return m == top ? 1.0f : ex2(m - top); }
__device__ __forceinline__ float paged_inverse(float sum, float scale) { return sum > 0 ? scale / sum : sum; }
__device__ __forceinline__ float paged_log_sum(float top, float sum) {
  return sum == 0 ? -INFINITY : (top + log2f(sum)) * 0.69314718055994530942f;
}

template <typename TQ, typename TC, int D, int NT>
__global__ void __launch_bounds__(PagedShape<TQ, TC, D, NT>::kThreads, 1) paged_kernel(const PagedArgs a) {
  using S = PagedShape<TQ, TC, D, NT>;
  using TM = typename S::TM;
  constexpr int kWarps = S::kWarps, kThreads = S::kThreads, kDepth = S::kDepth, kRow = S::kRow, kTile = S::kTile;
  constexpr int kSub = S::kSub, kTokens = S::kTokens;
  constexpr uint32_t kAll = kSub == 2 ? ~0u : 0xffffu;
  constexpr int kLead = 2 * kDepth - 1;    // copy groups that may be in flight behind the one that is waited for
  // weights up to 2^14 in fp16: it keeps 2^-38 of the largest
  constexpr float kLift = std::is_same<TM, __half>::value ? 14.0f : 0.0f;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int64_t s_scan[kWarps];
  __shared__ OpenState s_open[2 * kWarps];   // of a warp: of the unit it ends, of the unit it leaves unfinished
  __shared__ int s_last;
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

  // The tiles of all units; thread i sums those of its run of sequences.
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b_lo = min(tid * per, a.B), b_hi = min(b_lo + per, a.B);
  int64_t mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const TileRange t = tile_range<kTokens>(a, b);
    mine += max(0, t.end - t.first);
  }
  int64_t upto = mine;
#pragma unroll
  for (int w = 1; w < 32; w <<= 1) {
    const int64_t x = __shfl_up_sync(~0u, upto, w);
    if (lane >= w) upto += x;
  }
  if (lane == 31) s_scan[warp] = upto;
  s_open[tid % (2 * kWarps)].x1 = 0;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += s_scan[w];
  total *= units;
  const int G = static_cast<int>(min(static_cast<int64_t>(gridDim.x), max(int64_t{1}, total / (kWarps * a.min_tiles))));
  const int c = blockIdx.x;
  if (total == 0 || c >= G) return;
  // warp i of the G kWarps takes [first_of(i), first_of(i + 1))
  const int64_t quot = total / (G * kWarps);
  const int rem = static_cast<int>(total % (G * kWarps));
  const auto first_of = [&](int i) { return quot * i + min(i, rem); };
  const auto cta_of = [&](int64_t x) {
    const int64_t wide = rem * (quot + 1);
    return static_cast<int>(x < wide ? x / (quot + 1) : rem + (x - wide) / quot) / kWarps;
  };
  const int64_t f0 = first_of(c * kWarps), f1 = first_of((c + 1) * kWarps);
  const int64_t w0 = first_of(c * kWarps + warp), w1 = first_of(c * kWarps + warp + 1);

  if (w0 < w1) {
    // ---- where w0 lies: the run of sequences by the sums, then the sequence
    TileCursor seg;    // the unit being attended
    int64_t pre = 0;
    {
      int run = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {   // the run's warp
        if (w0 >= (pre + s_scan[w]) * units && w + 1 < kWarps && run == 32 * w) {
          pre += s_scan[w];
          run = 32 * (w + 1);
        }
      }
      // the run: lane i sums run i of that warp again
      const int lo = min((run + lane) * per, a.B), hi = min(lo + per, a.B);
      int64_t sum = 0;
      for (int b = lo; b < hi; ++b) {
        const TileRange t = tile_range<kTokens>(a, b);
        sum += max(0, t.end - t.first);
      }
      int64_t end = sum;
#pragma unroll
      for (int w = 1; w < 32; w <<= 1) {
        const int64_t x = __shfl_up_sync(~0u, end, w);
        if (lane >= w) end += x;
      }
      const int at = __ffs(__ballot_sync(~0u, w0 < (pre + end) * units)) - 1;
      pre += __shfl_sync(~0u, end - sum, at);
      seg.b = (run + at) * per;
      for (;; ++seg.b) {
        seg.t = tile_range<kTokens>(a, seg.b);
        const int n = max(0, seg.t.end - seg.t.first);
        if (w0 < (pre + n) * units) break;
        pre += n;
      }
      const int64_t off = w0 - pre * units;
      const int n = seg.t.end - seg.t.first;
      seg.u = static_cast<int>(off / n);
      seg.at = seg.t.first + static_cast<int>(off - static_cast<int64_t>(seg.u) * n);
    }

    // ---- loads
    unsigned char* const my_ring = smem + S::kRing + warp * S::kRingWarp;
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(my_ring));
    uint32_t* const masks = reinterpret_cast<uint32_t*>(smem + S::kMasks) + warp * kDepth;
    constexpr int kSize = static_cast<int>(sizeof(TC));
    constexpr int kChunks = kRow / 16;               // 16-byte chunks of a row
    constexpr int kRows = kChunks >= 32 ? 1 : 32 / kChunks;   // rows of a warp's copy
    constexpr int kCopies = kTokens / kRows;
    const int row0 = lane / kChunks, chunk0 = lane % kChunks;
    const bool whole = (a.page & 15) == 0;           // 16 rows do not cross pages
    const unsigned char* const Kb = static_cast<const unsigned char*>(a.K) + chunk0 * 16;
    const unsigned char* const Vb = static_cast<const unsigned char*>(a.V) + chunk0 * 16;
    TileCursor ld = seg;
    int64_t ld_left = w1 - w0;   // tiles that have not been asked for
    const unsigned char *Kh = Kb, *Vh = Vb;   // of the tile's KV head
    int id = 0, in_page = 0;     // of the tile's row `lane` (of the first of its 16 rows, if whole)
    uint32_t mask = 0;           // the tile's rows that are tokens
    uint32_t live = 0;           // of these, those in a page of the pool
    const auto find = [&]() {    // the tile at ld
      const int row = ld.at * kTokens + (lane & (kTokens - 1));
      const bool in = row >= ld.t.lo && row < ld.t.len;
      const int n = whole ? row & ~15 : row;
      const int p = page_of(a, n);
      in_page = n - p * a.page;
      id = 0;
      // a 16-row product without tokens (behind the last, before the window) has no page of its own
      const uint32_t rows = __ballot_sync(~0u, in);
      const bool ask = whole ? ((rows >> (lane & 16)) & 0xffffu) != 0 : in;
      if (ask) id = a.table[static_cast<int64_t>(ld.b) * a.table_stride + p];
      mask = rows & kAll;
      const int kv = a.chunks == 1 ? ld.u : ld.u / a.chunks;
      Kh = Kb + kv * a.k_head * kSize;
      Vh = Vb + kv * a.v_head * kSize;
    };
    const auto copy_rows = [&](uint32_t dst, const unsigned char* base, int64_t page, int64_t tok) {
      if (whole) {
#pragma unroll
        for (int m = 0; m < kSub; ++m) {
          const int64_t mid = kSub == 1 ? id : __shfl_sync(~0u, id, 16 * m);
          const int64_t min_page = kSub == 1 ? in_page : __shfl_sync(~0u, in_page, 16 * m);
          const unsigned char* src = base + (mid * page + (min_page + row0) * tok) * kSize;
          const int64_t step = tok * (kRows * kSize);
          const bool full = ((live >> (16 * m)) & 0xffffu) == 0xffffu;
#pragma unroll
          for (int j = 0; j < kCopies / kSub; ++j) {
            const int row = m * 16 + j * kRows + row0;
            copy16(dst + swizzled<kRow>(row, chunk0), src, full || ((live >> row) & 1));
            src += step;
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < kCopies; ++j) {
          const int row = j * kRows + row0;
          const int64_t rid = __shfl_sync(~0u, id, row), rin = __shfl_sync(~0u, in_page, row);
          const bool on = (live >> row) & 1;
          copy16(dst + swizzled<kRow>(row, chunk0), on ? base + (rid * page + rin * tok) * kSize : base, on);
        }
      }
    };
    // K, then V, of the tile at ld go to a slot; the two calls of a tile stand around the products of another
    const auto issue_k = [&](int slot) {
      if (ld_left > 0) {
        const bool ok = static_cast<uint32_t>(id) < static_cast<uint32_t>(a.n_pages);
        live = mask & __ballot_sync(~0u, ok);
        if (!ok) id = 0;
        if (lane == 0) {
          masks[slot] = live;
          if (live != mask) *a.status = HHR_ERR_BAD_INDEX;
        }
        copy_rows(ring + slot * 2 * kTile, Kh, a.k_page, a.k_tok);
      }
      copy_commit();
    };
    const auto issue_v = [&](int slot) {
      if (ld_left > 0) {
        copy_rows(ring + slot * 2 * kTile + kTile, Vh, a.v_page, a.v_tok);
        if (--ld_left > 0) {
          ld.next<kTokens>(a, units);
          find();
        }
      }
      copy_commit();
    };
    find();
#pragma unroll 1
    for (int s = 0; s < kDepth; ++s) {
      issue_k(s);
      issue_v(s);
    }

    unsigned char* const my_q = smem + S::kQ + warp * S::kQWarp;
    const uint32_t q_smem = static_cast<uint32_t>(__cvta_generic_to_shared(my_q));
    int slot = 0;
    int64_t f = w0;

    while (true) {   // units of this warp's range
      const int g_kv = seg.u / a.chunks, first_head = (seg.u - g_kv * a.chunks) * a.chunk;
      const int heads = min(a.chunk, a.r - first_head);
      const int head0 = g_kv * a.r + first_head;
      const int64_t x0 = f - (seg.at - seg.t.first), x1 = x0 + (seg.t.end - seg.t.first);
      const bool began = f == x0, ends = x1 <= w1;
      int left = static_cast<int>((ends ? x1 : w1) - f);

      // Queries: lane (g, t4) holds elements 2 t4, 2 t4 + 1 and 8 + 2 t4, 9 + 2 t4 of every 16 of head g; with 8-bit keys
      // 4 t4 .. 4 t4 + 3, the order in which the bytes of a row fill their fragments.
      uint32_t qf[D / 16][NT][2];
      float sc[NT][2], m[NT][2], base[NT][2], l[NT][2], o[NT][D / 16][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const bool on = n * 8 + g < heads;
        const TQ* const row = static_cast<const TQ*>(a.q) + seg.b * a.q_seq + static_cast<int64_t>(head0 + (on ? n * 8 + g : 0)) * D;
        float up = a.scale_log2;
        if constexpr (std::is_same<TQ, TM>::value) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            if constexpr (S::kE4) {
              const uint2 x = *reinterpret_cast<const uint2*>(row + k * 16 + 4 * t4);
              qf[k][n][0] = on ? x.x : 0;
              qf[k][n][1] = on ? x.y : 0;
            } else {
              const uint32_t x = *reinterpret_cast<const uint32_t*>(row + k * 16 + 2 * t4);
              const uint32_t y = *reinterpret_cast<const uint32_t*>(row + k * 16 + 8 + 2 * t4);
              qf[k][n][0] = on ? x : 0;
              qf[k][n][1] = on ? y : 0;
            }
          }
        } else {   // bf16 queries of an 8-bit cache
          float top = 0;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint2 x = *reinterpret_cast<const uint2*>(row + k * 16 + 4 * t4);
            qf[k][n][0] = on ? x.x : 0;
            qf[k][n][1] = on ? x.y : 0;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qf[k][n][e]));
              top = fmaxf(top, fmaxf(fabsf(y.x), fabsf(y.y)));
            }
          }
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
          top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
          const int by = top > 0 && top < INFINITY ? 14 - ilogbf(top) : 0;
          const float one = ldexpf(1.0f, by / 2), two = ldexpf(1.0f, by - by / 2);   // 2^by may be beyond float
          up = ldexpf(up, -by);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qf[k][n][e]));
              const __half2 h = __floats2half2_rn(y.x * one * two, y.y * one * two);
              qf[k][n][e] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sc[n][e] = __shfl_sync(~0u, up, (2 * t4 + e) * 4);
          m[n][e] = -INFINITY;
          base[n][e] = l[n][e] = 0;
        }
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][j][e] = 0;
      }
      if constexpr (!S::kQRegs) {   // as fragments: 8 bytes a lane
        __syncwarp();
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int n = 0; n < NT; ++n)
            *reinterpret_cast<uint2*>(my_q + ((k * NT + n) * 32 + lane) * 8) = make_uint2(qf[k][n][0], qf[k][n][1]);
        __syncwarp();
      }

      f += left;
      for (; left > 0; --left) {
        const uint32_t kt = ring + slot * 2 * kTile, vt = kt + kTile;
        copy_wait<kLead>();
        __syncwarp();
        const uint32_t rows = masks[slot];
        // S^T = K Q^T; a lone product in two sums, so that its steps wait less for one another
        constexpr int kSums = kSub == 1 ? 2 : 1;
        float s[kSub][kSums][NT][4];
#pragma unroll
        for (int i = 0; i < kSub; ++i)
#pragma unroll
          for (int h = 0; h < kSums; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[i][h][n][e] = 0;
        const auto dot = [&](int i, int k, const uint32_t (&r)[4]) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            uint2 q;
            if constexpr (S::kQRegs)
              q = make_uint2(qf[k][n][0], qf[k][n][1]);
            else
              q = *reinterpret_cast<const uint2*>(my_q + ((k * NT + n) * 32 + lane) * 8);
            mma<TM>(s[i][k % kSums][n], r, q.x, q.y);
          }
        };
#pragma unroll
        for (int k = 0; k < D / 16; k += S::kE4 ? 2 : 1)
#pragma unroll
          for (int i = 0; i < kSub; ++i) {
            uint32_t r[4];
            ldsm4(r, kt + swizzled<kRow>(i * 16 + (lane & 15), (S::kE4 ? k : 2 * k) + (lane >> 4)));
            if constexpr (S::kE4) {
              dot(i, k, {wide_lo(r[0]), wide_lo(r[1]), wide_hi(r[0]), wide_hi(r[1])});
              dot(i, k + 1, {wide_lo(r[2]), wide_lo(r[3]), wide_hi(r[2]), wide_hi(r[3])});
            } else {
              dot(i, k, r);
            }
          }
        __syncwarp();
        issue_k(slot);
        // weights: lane (g, t4) holds tokens g and g + 8 of heads 2 t4 and 2 t4 + 1
        bool grown = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < kSub; ++i) {
            float(&x)[4] = s[i][0][n];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = (kSums == 2 ? x[e] + s[i][kSums - 1][n][e] : x[e]) * sc[n][e & 1];
            if (rows != kAll) {
              if (!((rows >> (16 * i + g)) & 1)) x[0] = x[1] = -INFINITY;
              if (!((rows >> (16 * i + g + 8)) & 1)) x[2] = x[3] = -INFINITY;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) grown = grown || fmaxf(x[e], x[e + 2]) > m[n][e];
          }
        if (__any_sync(~0u, grown)) {   // rare after the first tiles
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float top = m[n][e];
#pragma unroll
              for (int i = 0; i < kSub; ++i) top = fmaxf(top, fmaxf(s[i][0][n][e], s[i][0][n][e + 2]));
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
        uint32_t hi[kSub][NT][2], lo[kSub][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < kSub; ++i) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = ex2(s[i][0][n][e] - base[n][e & 1]);
            l[n][0] += w[0] + w[2];
            l[n][1] += w[1] + w[3];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              split<TM>(w[2 * e], w[2 * e + 1], hi[i][n][e], lo[i][n][e]);
              hi[i][n][e] = transposed(hi[i][n][e]);
              lo[i][n][e] = transposed(lo[i][n][e]);
            }
          }
        copy_wait<kLead>();
        __syncwarp();
        // O^T += V^T P^T
#pragma unroll
        for (int j = 0; j < D / 16; j += S::kE4 ? 2 : 1)
#pragma unroll
          for (int i = 0; i < kSub; ++i) {
            const auto add = [&](int to, const uint32_t (&r)[4]) {
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                mma<TM>(o[n][to], r, hi[i][n][0], hi[i][n][1]);
                mma<TM>(o[n][to], r, lo[i][n][0], lo[i][n][1]);
              }
            };
            uint32_t r[4];
            if constexpr (S::kE4) {
              // a transposed 2-byte element is columns 2 g and 2 g + 1 of a token: rows g and g + 8 of the product
              ldsm4_trans(r, vt + swizzled<kRow>(i * 16 + (lane & 15), j + (lane >> 4)));
#pragma unroll
              for (int e = 0; e < 4; ++e) r[e] = __byte_perm(r[e], 0, 0x3120);
              add(j, {wide_lo(r[0]), wide_hi(r[0]), wide_lo(r[1]), wide_hi(r[1])});
              add(j + 1, {wide_lo(r[2]), wide_hi(r[2]), wide_lo(r[3]), wide_hi(r[3])});
            } else {
              ldsm4_trans(r, vt + swizzled<kRow>(i * 16 + (lane & 7) + (lane >> 4) * 8, 2 * j + ((lane >> 3) & 1)));
              add(j, r);
            }
          }
        __syncwarp();
        issue_v(slot);
        slot = slot + 1 == kDepth ? 0 : slot + 1;
      }

      // ---- the unit ends here, or the range does
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) l[n][e] += __shfl_xor_sync(~0u, l[n][e], w);
      if (began && ends) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int h = n * 8 + 2 * t4 + e;
            if (h >= heads) continue;
            const float inv = paged_inverse(l[n][e], a.v_scale);
            const size_t row = static_cast<size_t>(seg.b) * a.Hq + head0 + h;
            if (a.lse && g == 0) a.lse[row] = paged_log_sum(base[n][e], l[n][e]);
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int d = j * 16 + (S::kE4 ? 2 * g + i : g + 8 * i);
                if (a.out_f32)
                  static_cast<float*>(a.out)[row * D + d] = o[n][j][e + 2 * i] * inv;
                else
                  static_cast<TQ*>(a.out)[row * D + d] = from_f32<TQ>(o[n][j][e + 2 * i] * inv);
              }
          }
      } else {
        // the last one may lie over the warp's ring, which is drained
        const bool last = f == w1;
        float* const to = last ? reinterpret_cast<float*>(my_ring) : a.firsts + static_cast<size_t>(c * kWarps + warp) * a.state;
        if (last) __syncwarp();
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int h = n * 8 + 2 * t4 + e;
            if (h >= heads) continue;
            float* const row = to + h * (D + 4);
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              if constexpr (S::kE4) {
                *reinterpret_cast<float2*>(row + j * 16 + 2 * g) = make_float2(o[n][j][e], o[n][j][e + 2]);
              } else {
                row[j * 16 + g] = o[n][j][e];
                row[j * 16 + g + 8] = o[n][j][e + 2];
              }
            }
            if (g == 0) *reinterpret_cast<float2*>(row + D) = make_float2(m[n][e] == -INFINITY ? -INFINITY : base[n][e], l[n][e]);
          }
        if (lane == 0) s_open[2 * warp + last] = {x0, x1, to, seg.b, seg.u};
      }
      if (f == w1) break;
      seg.at = seg.t.end - 1;
      seg.next<kTokens>(a, units);
    }
  }
  __syncthreads();

  // ---- open states, in the order of the tokens: those of one unit are joined
  const auto finish = [&](size_t at, float4 y, float inv) {   // four columns
    if (a.out_f32) {
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
    } else {
      Pack<TQ, 4> p;
      p.v[0] = from_f32<TQ>(y.x * inv);
      p.v[1] = from_f32<TQ>(y.y * inv);
      p.v[2] = from_f32<TQ>(y.z * inv);
      p.v[3] = from_f32<TQ>(y.w * inv);
      *reinterpret_cast<Pack<TQ, 4>*>(static_cast<TQ*>(a.out) + at) = p;
    }
  };
  for (int i0 = 0, i1; i0 < 2 * kWarps; i0 = i1) {
    i1 = i0 + 1;
    const int64_t x0 = s_open[i0].x0, x1 = s_open[i0].x1;
    if (x1 == 0) continue;
    int states = 1;
    uint32_t which = 1u << i0;
    while (i1 < 2 * kWarps && (s_open[i1].x1 == 0 || s_open[i1].x0 == x0)) {
      if (s_open[i1].x1) {
        which |= 1u << i1;
        ++states;
      }
      ++i1;
    }
    const int b = s_open[i0].b, u = s_open[i0].u;
    const int g_kv = u / a.chunks, first_head = (u - g_kv * a.chunks) * a.chunk;
    const int heads = min(a.chunk, a.r - first_head);
    const size_t out_row = static_cast<size_t>(b) * a.Hq + g_kv * a.r + first_head;
    const bool inside = x0 >= f0 && x1 <= f1;
    const int c0 = inside ? c : cta_of(x0);
    float* const part = a.parts + static_cast<size_t>(2 * c + (c == c0)) * a.state;
    for (int e = tid; e < heads * (D / 4); e += kThreads) {
      const int h = e / (D / 4), d = e % (D / 4) * 4;
      float top = -INFINITY, sum = 0;
      for (uint32_t w = which; w; w &= w - 1) top = fmaxf(top, s_open[__ffs(w) - 1].at[h * (D + 4) + D]);
      float4 y = make_float4(0, 0, 0, 0);
      for (uint32_t w = which; w; w &= w - 1) {
        const float* const row = s_open[__ffs(w) - 1].at + h * (D + 4);
        const float2 ml = *reinterpret_cast<const float2*>(row + D);
        const float4 x = *reinterpret_cast<const float4*>(row + d);
        const float by = paged_weight(ml.x, top);
        sum = fmaf(ml.y, by, sum);
        y.x = fmaf(x.x, by, y.x);
        y.y = fmaf(x.y, by, y.y);
        y.z = fmaf(x.z, by, y.z);
        y.w = fmaf(x.w, by, y.w);
      }
      if (inside) {
        finish((out_row + h) * D + d, y, paged_inverse(sum, a.v_scale));
        if (d == 0 && a.lse) a.lse[out_row + h] = paged_log_sum(top, sum);
      } else {
        *reinterpret_cast<float4*>(part + h * (D + 4) + d) = y;
        if (d == 0) *reinterpret_cast<float2*>(part + h * (D + 4) + D) = make_float2(top, sum);
      }
    }
    if (inside) continue;

    // The last of the unit's CTAs to arrive joins their states from L2.
    const int n_parts = cta_of(x1 - 1) - c0 + 1;
    __syncthreads();
    if (tid == 0) {
      __threadfence();
      const bool last = atomicAdd(a.counters + c0, 1u) == static_cast<uint32_t>(n_parts - 1);
      if (last) a.counters[c0] = 0;
      __threadfence();
      s_last = last;
    }
    __syncthreads();
    if (!s_last) continue;
    float* const by = reinterpret_cast<float*>(smem + S::kQ);   // [8][n_parts]
    float* const invs = by + 8 * kPagedMaxGrid;                 // [8]
    float4* const sums = reinterpret_cast<float4*>(invs + 8);   // [kThreads]
    const auto part_of = [&](int i) { return a.parts + static_cast<size_t>(2 * (c0 + i) + (i == 0)) * a.state; };
    for (int h0 = 0; h0 < heads; h0 += 8) {
      const int n_heads = min(8, heads - h0);
      for (int h = warp; h < n_heads; h += kWarps) {
        float top = -INFINITY, sum = 0;
        for (int i = lane; i < n_parts; i += 32) top = fmaxf(top, __ldcg(part_of(i) + (h0 + h) * (D + 4) + D));
#pragma unroll
        for (int w = 16; w; w >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, w));
        for (int i = lane; i < n_parts; i += 32) {
          const float2 ml = __ldcg(reinterpret_cast<const float2*>(part_of(i) + (h0 + h) * (D + 4) + D));
          const float x = paged_weight(ml.x, top);
          by[h * n_parts + i] = x;
          sum = fmaf(ml.y, x, sum);
        }
#pragma unroll
        for (int w = 16; w; w >>= 1) sum += __shfl_xor_sync(~0u, sum, w);
        if (lane == 0) {
          invs[h] = paged_inverse(sum, a.v_scale);
          if (a.lse) a.lse[out_row + h0 + h] = paged_log_sum(top, sum);
        }
      }
      __syncthreads();
      const int items = n_heads * (D / 4);                 // 4 columns each
      const int splits = max(1, kThreads / items);         // parts are dealt out where there are few items
      for (int e0 = 0; e0 < items; e0 += kThreads) {
        const int e = splits > 1 ? tid % items : e0 + tid, sp = splits > 1 ? tid / items : 0;
        const int h = e / (D / 4), d = e % (D / 4) * 4;
        float4 y = make_float4(0, 0, 0, 0);
        if (e < items && sp < splits) {
#pragma unroll 8
          for (int i = sp; i < n_parts; i += splits) {
            const float4 x = __ldcg(reinterpret_cast<const float4*>(part_of(i) + (h0 + h) * (D + 4) + d));
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
        if (e < items && sp == 0) finish((out_row + h0 + h) * D + d, y, invs[h]);
      }
      __syncthreads();
    }
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
