// The kernel of hhr_paged_attend: attention of one new token per sequence over
// a paged key-value cache, split over the cache's length and joined.
//
// out[h] = sum_n w_n V[n] / sum_n w_n with w_n = 2^((x_n - m) c), x_n = q[h].K[n], c = scale log2(e), m the largest x_n:
// one pass over K and V with a running m, rescaling what was summed whenever m grows; states of disjoint token ranges
// (m, sum w, sum w V) join by rescaling to the larger m.  The difference is taken before the scale: it rounds at its own
// size and not at the logits', and a mask by a type's lowest value cannot overflow on the way.
//
// Bound: HBM.  A token costs 2 d elements of K and V per KV head and 4 d r operations for its r query heads: 2 to 24
// operations per byte, far below what the tensor cores do in that time, so the work is to keep loads in flight.
//
// Work.  A unit is (sequence, KV head, chunk of its query heads); its tokens are cut into tiles of 16 or 32.  The tiles
// of all units, one after another, are dealt out evenly: every warp of the card takes a contiguous range, so it ends one
// unit, does some whole ones and begins one, whatever the lengths are.  Lengths are read on the device (a captured call
// follows them).  A whole unit is written by its warp alone; the states of a unit that several warps share are joined by
// their CTA when its warps are done, and by the last of its CTAs to arrive if it has several: always in the same
// order, so the result does not depend on which one that is.  Only a CTA's first and last unit are shared with its
// neighbours: the workspace is for the card's CTAs and not for the sequences.  No CTA waits for another.
//
// Tiles.  Each warp copies its tiles into its own ring (cp.async, 16 bytes a lane, swizzled) kDepth tiles ahead, across
// the borders of units: no barrier stands anywhere before the join, and loads go on while a unit ends.  Rows are
// addressed one by one through the table, which takes any page size; where a page holds whole 16-row tiles one table
// entry serves all of them.
//
// Products.  S^T = K Q^T (m16n8k16, tokens by heads: 8 heads fill n where a tile of 16 query rows would be half empty)
// and O^T += V^T P^T, float32 sums.  P is a sum of 16-bit terms, by what the output's own rounding hides: three of bf16
// for a float32 output (2^-25), two of bf16 for a bf16 output (2^-17; one, 2^-8, would show; three change 0.3 % of the
// values by a step and cost 8 % in groups of 12 to 24 heads), two of fp16 (2^-22; one, 2^-11, is an eighth of a bf16
// output's rounding, but moves 6 % of its values a step from the float32 result's rounding where two move 0.1 %; it takes
// 53 us where two take 59, 16 heads, 8-bit cache).  The tensor cores' own sums lose up to a few units of their last place
// at every step, all in one direction: a tile's product is a sum of its own, added by an ordinary addition (a warp's unit
// of 64K tokens: relative error 4e-6; in the tensor cores 2.9e-4, half a step of fp16; groups of up to 8 heads take the
// same time, 16 heads of an 8-bit cache 61 us for 60, 24 heads of bf16 54 for 51).  8-bit elements become fp16 in
// registers, exactly; bf16 queries of an 8-bit cache become fp16 after a power of two per row that makes their largest
// element about 2^14 (elements below 2^-28 of it lose bits).  mma.sync and not tcgen05: a tile is 16 tokens of one warp,
// whose P never leaves its registers; the tensor pipe has room to spare (busy 18 % at 128K), and a 128-row tile with its
// commits would couple the warps that the private rings keep apart.
//
// Measured (B200, captured passes): 1 x 128K, 8 KV heads of 128, bf16: 87 us, 6.2 TB/s (0.95 of the copy bandwidth);
// 8 x 64K: 305 to 312 us by the GPU, 6.9 to 7.0 TB/s; 61 ragged sequences to 8191, groups of 8, fp16: 119 us, 5.5 TB/s;
// 16 ragged to 32K, 4 KV heads, groups of 16, e4m3: 61 us, 2.45 TB/s (issue and latency of the conversions and products,
// then the joins); one sequence of 517: 10 us (latency, and the launch arguments that every thread copies to local memory
// for the join, 12.7 MB a call).  DRAM reads are 1.00 of the keys and values.
#pragma once

#include <algorithm>
#include <type_traits>

#include "hhr_internal.cuh"
#include "paged_common.cuh"
#include "paged_tiles.cuh"

namespace hhr {

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
  // Registers hold the query fragments of 8 heads; those of more are read from shared memory, each warp its own copy
  // (16 heads, d = 128, 8-bit, one term a weight: 58 us in registers of 8 warps, 55 of 12 warps, 53 from shared memory;
  // the variants of 16 and more heads spill 4 to 56 bytes a thread all the same).
  static constexpr bool kQRegs = NT == 1;
  // More warps hide more latency where their registers allow it.  The rings together hold about 100 KB: with 192 KB in
  // flight the SMs at the head of their group run 25 % ahead of the last ones and the call waits for those (8 sequences
  // of 64K, 8 KV heads, bf16: 340 us with 192 KB, 326 with 128, 324 with 64 in 8 warps; 312 with 96 KB in 12 warps).
  static constexpr int kWarps = D < 256 && NT <= 2 ? 12 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kDepth = std::max(1, 131072 / (kWarps * 2 * kTile));
  // shared memory
  static constexpr int kRing = 0;
  // of a warp; in the end it holds the warp's last state
  static constexpr int kRingWarp = std::max(kDepth * 2 * kTile, (kHeads * (D + 4) * 4 + 127) / 128 * 128);
  static constexpr int kQ = kRing + kWarps * kRingWarp;
  static constexpr int kQWarp = kQRegs ? 0 : kHeads * D * 2;
  static constexpr int kMasks = kQ + kWarps * kQWarp;
  static constexpr int kSmem = kMasks + kWarps * kDepth * 4;
  static_assert(kSmem <= 226 * 1024, "shared memory of a CTA");
};

__device__ __forceinline__ int page_of(const PagedArgs& a, int n) {
  return static_cast<int>((__umulhi(static_cast<uint32_t>(n), a.page_magic) + static_cast<uint32_t>(n)) >> a.page_shift);
}

// An open state: one of several of its unit.
struct OpenState {
  int64_t x0, x1;       // the unit's tiles; x1 = 0: none
  int b, u;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Copies of K and V: read once, so L2 lets them go first and keeps tables, exchanged states and code.
__device__ __forceinline__ uint64_t read_once() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint64_t policy, bool live) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0),
               "l"(policy)
               : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy) : "memory");
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

// Two floats as pairs of 16-bit values, one for each term: every one rounds what those before it leave.
template <typename TM, int kTerms>
__device__ __forceinline__ void split(float x, float y, uint32_t (&term)[kTerms]) {
#pragma unroll
  for (int k = 0; k < kTerms; ++k) {
    if constexpr (std::is_same<TM, __half>::value) {
      const __half2 h = __floats2half2_rn(x, y);
      term[k] = *reinterpret_cast<const uint32_t*>(&h);
      const float2 f = __half22float2(h);
      x -= f.x;
      y -= f.y;
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
      term[k] = *reinterpret_cast<const uint32_t*>(&h);
      const float2 f = __bfloat1622float2(h);
      x -= f.x;
      y -= f.y;
    }
  }
}

// Four e4m3 values as fp16, exactly: the low and the high pair.  (The header's conversion of a pair goes through two
// 16-bit halves and takes 3.6 cycles an SM for four values, this form 1.5.)
__device__ __forceinline__ void widen(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\ncvt.rn.f16x2.e4m3x2 %0, l;\ncvt.rn.f16x2.e4m3x2 %1, h;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}

// Tiles lie in shared memory as rows of `row` bytes whose 16-byte chunk c stands at c ^ (i & 7) in row i (at
// c ^ ((i >> 1) & 3) in rows of 64 bytes): eight rows read at the same chunk, or one row's chunks, fall on different
// banks.  The lowest bits of a row and a chunk go through turn(); the rest of both are added, so that the addresses of a
// tile differ from a few lane-owned ones by constants.
template <int row>
__device__ __forceinline__ int turn(int i, int c) {
  return i * row + ((c ^ (row >= 128 ? (i & 7) : ((i >> 1) & 3))) << 4);
}
template <int row>
__device__ __forceinline__ uint32_t chunk_at(uint32_t turned, int c) {   // turned + chunk c, where turned has chunk 0 or 1
  return (turned ^ ((c & 7) << 4)) + (c >> 3) * 128;
}

// The maximum of a state is exchanged as a quarter of its logit in powers of two: a finite logit times log2(e) may be
// beyond float32.  The weight of a state of maximum m among states of maximum top; 1 / sum of a unit's weights (0 for
// none, NaN stays) and its log-sum-exp, where the weights are 2^lift times what they stand for.
__device__ __forceinline__ float paged_quarter(float m, float scale) { return m == -INFINITY ? m : m * (scale * 0.25f); }
__device__ __forceinline__ float paged_weight(float m, float top) { return m == top ? 1.0f : ex2((m - top) * 4.0f); }
__device__ __forceinline__ float paged_inverse(float sum, float scale) { return sum > 0 ? scale / sum : sum; }
__device__ __forceinline__ float paged_log_sum(float top, float sum, float lift) {
  constexpr float kLn2 = 0.69314718055994530942f;
  return sum == 0 ? -INFINITY : fmaf(top, 4.0f * kLn2, (log2f(sum) - lift) * kLn2);
}

// Weights of fp16 terms are lifted to 2^14 at most: fp16 keeps 2^-38 of the largest.  The lift is added to a difference
// from the largest (it rounds to 2^-21 there): subtracted from the largest logit it would round at the logit's size, to
// 16 and a weight beyond fp16 where logits reach 2^25.
template <typename TM>
__device__ constexpr float kPagedLift = std::is_same<TM, __half>::value ? 14.0f : 0.0f;

// A join of n states: the i-th at base + i * stride, the last at `last` unless that is null; into the state `to` (none of
// these), or, if that is null, into the output's rows from out_row on.
struct Join {
  const float* base;
  const float* last;
  float* to;
  size_t out_row;
  int64_t x0, x1;       // the unit's tiles
  int stride, n, heads;
};

// All threads of a CTA do `count` joins side by side, a thread four columns of a head at a time.  One copy of this code
// serves all joins: it is fetched cold.
template <typename TQ, typename TM, int D, int kThreads>
__device__ __noinline__ void join_states(const PagedArgs& a, const Join* joins, int count) {
  const int most = a.chunk * (D / 4);
#pragma unroll 1
  for (int e = threadIdx.x; e < count * most; e += kThreads) {
    const int k = e / most, item = e - k * most, h = item / (D / 4), d = item % (D / 4) * 4;
    const Join& j = joins[k];
    const int n = j.n;
    if (h >= j.heads) continue;
    const float* const base = j.base + h * (D + 4);
    const int stride = j.stride;
    const float* const last = j.last ? j.last + h * (D + 4) : base + (n - 1) * stride;
    float top = -INFINITY, sum = 0;
    float4 y = make_float4(0, 0, 0, 0);
    constexpr int kBatch = 8;    // loads in flight: the states may lie in L2
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += kBatch) {
      float2 ml[kBatch];
      float4 x[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        ml[k] = make_float2(-INFINITY, 0);
        x[k] = make_float4(0, 0, 0, 0);
        if (i0 + k < n) {
          const float* const row = i0 + k < n - 1 ? base + (i0 + k) * stride : last;
          ml[k] = *reinterpret_cast<const float2*>(row + D);
          x[k] = *reinterpret_cast<const float4*>(row + d);
        }
      }
      float next = top;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) next = fmaxf(next, ml[k].x);
      const float was = paged_weight(top, next);
      sum *= was;
      y = make_float4(y.x * was, y.y * was, y.z * was, y.w * was);
      top = next;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float by = paged_weight(ml[k].x, top);
        sum = fmaf(ml[k].y, by, sum);
        y.x = fmaf(x[k].x, by, y.x);
        y.y = fmaf(x[k].y, by, y.y);
        y.z = fmaf(x[k].z, by, y.z);
        y.w = fmaf(x[k].w, by, y.w);
      }
    }
    if (j.to) {
      *reinterpret_cast<float4*>(j.to + h * (D + 4) + d) = y;
      if (d == 0) *reinterpret_cast<float2*>(j.to + h * (D + 4) + D) = make_float2(top, sum);
      continue;
    }
    const float inv = paged_inverse(sum, a.v_scale);
    const size_t at = (j.out_row + h) * D + d;
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
    if (d == 0 && a.lse) a.lse[j.out_row + h] = paged_log_sum(top, sum, kPagedLift<TM>);
  }
}

// kFine: bf16 products for a float32 output.
template <typename TQ, typename TC, int D, int NT, bool kFine>
__global__ void __launch_bounds__(PagedShape<TQ, TC, D, NT>::kThreads, 1) paged_kernel(const PagedArgs a) {
  using S = PagedShape<TQ, TC, D, NT>;
  using TM = typename S::TM;
  constexpr int kWarps = S::kWarps, kThreads = S::kThreads, kDepth = S::kDepth, kRow = S::kRow, kTile = S::kTile;
  constexpr int kSub = S::kSub, kTokens = S::kTokens;
  constexpr uint32_t kAll = kSub == 2 ? ~0u : 0xffffu;
  constexpr int kTerms = kFine ? 3 : 2;    // of a weight (see the head of this file)
  constexpr int kLead = 2 * kDepth - 1;    // copy groups that may be in flight behind the one that is waited for
  constexpr float kLift = kPagedLift<TM>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int64_t s_scan[kWarps], s_before[kThreads];
  __shared__ Join s_join[kWarps + 1];
  __shared__ int s_joins, s_side[2];                  // joins; those of the units shared with the CTAs before and behind
  __shared__ int s_last[2];                           // of these: whether this CTA joins the CTAs' states
  __shared__ int s_seqs[kWarps];
  __shared__ OpenState s_open[2 * kWarps];   // of a warp: of the unit it ends, of the unit it leaves unfinished
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int units = a.Hkv * a.chunks;

  dependency_wait();
  launch_dependents();

  // The tiles before each run of `per` sequences: in the lanes of every warp where 32 hold them, or in shared memory.
  const bool few = a.B <= 32;
  const int per = few ? 1 : (a.B + kThreads - 1) / kThreads;
  int64_t total, before = 0;
  int n_seqs;          // sequences with tokens
  if (few) {
    int mine = 0;
    if (lane < a.B) {
      const TileRange t = tile_range<kTokens>(a, lane);
      mine = max(0, t.end - t.first);
    }
    int64_t upto = mine;
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
      const int64_t x = __shfl_up_sync(~0u, upto, w);
      if (lane >= w) upto += x;
    }
    total = __shfl_sync(~0u, upto, 31);
    before = upto - mine;
    n_seqs = __popc(__ballot_sync(~0u, mine > 0));
  } else {
    const int b_lo = min(tid * per, a.B), b_hi = min(b_lo + per, a.B);
    int64_t mine = 0;
    int seqs = 0;
    for (int b = b_lo; b < b_hi; ++b) {
      const TileRange t = tile_range<kTokens>(a, b);
      mine += max(0, t.end - t.first);
      seqs += t.end > t.first;
    }
    int64_t upto = mine;
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
      const int64_t x = __shfl_up_sync(~0u, upto, w);
      if (lane >= w) upto += x;
    }
    seqs = __reduce_add_sync(~0u, seqs);
    if (lane == 31) {
      s_scan[warp] = upto;
      s_seqs[warp] = seqs;
    }
    __syncthreads();
    total = 0;
    n_seqs = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) upto += s_scan[w];
      total += s_scan[w];
      n_seqs += s_seqs[w];
    }
    s_before[tid] = upto - mine;
  }
  if (tid < 2 * kWarps) s_open[tid].x1 = 0;
  __syncthreads();
  total *= units;
  // G CTAs take part with n_active warps each.  Where the tiles do not fill the card, G is a multiple of the units, so
  // that units of one length are not shared by CTAs (calls: 43 sequences of 3 tokens, 2 KV heads 9 us, with the tiles
  // packed into few CTAs 16; 9 sequences, window 128, 2 KV heads, groups of 24 25 us, with units shared 30).
  const int64_t n_units = static_cast<int64_t>(n_seqs) * units;
  const int64_t fill = total / (kWarps * a.min_tiles);
  const int G = static_cast<int>(fill >= gridDim.x || n_units > gridDim.x
                                     ? min(static_cast<int64_t>(gridDim.x), max(int64_t{1}, total))
                                     : max(int64_t{1}, max(int64_t{1}, fill / max(int64_t{1}, n_units)) * n_units));
  const int n_active = static_cast<int>(min(static_cast<int64_t>(kWarps), max(int64_t{1}, total / G)));
  const int c = blockIdx.x;
  // (a tile at least for each warp: the host bounds total * n_warps)
  const TileDeal deal(total, G, n_active);
  const int64_t f0 = deal.first_of(c * n_active), f1 = deal.first_of((c + 1) * n_active);
  const int64_t w0 = deal.first_of(c * n_active + warp), w1 = warp < n_active ? deal.first_of(c * n_active + warp + 1) : w0;

  if (w0 < w1) {
    // ---- where w0 lies: the last run that begins at or before it, then the sequence
    TileCursor seg;    // the unit being attended
    {
      int64_t pre;
      if (few) {
        seg.b = __popc(__ballot_sync(~0u, before * units <= w0)) - 1;
        pre = __shfl_sync(~0u, before, seg.b);
      } else {
        int run = -1;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) run += __popc(__ballot_sync(~0u, s_before[32 * w + lane] * units <= w0));
        pre = s_before[run];
        seg.b = run * per;
      }
      for (;; ++seg.b) {
        seg.t = tile_range<kTokens>(a, seg.b);
        const int n = max(0, seg.t.end - seg.t.first);
        if (w0 < (pre + n) * units || seg.b + 1 >= a.B) break;
        pre += n;
      }
      seg.place(w0 - pre * units, units);
    }

    // ---- loads
    unsigned char* const my_ring = smem + S::kRing + warp * S::kRingWarp;
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(my_ring));
    uint32_t* const masks = reinterpret_cast<uint32_t*>(smem + S::kMasks) + warp * kDepth;
    constexpr int kChunks = kRow / 16;               // 16-byte chunks of a row
    constexpr int kRows = kChunks >= 32 ? 1 : 32 / kChunks;   // rows of a warp's copy
    constexpr int kCopies = kTokens / kRows;
    const int row0 = lane / kChunks, chunk0 = lane % kChunks;
    const bool whole = (a.page & 15) == 0;           // 16 rows do not cross pages
    const unsigned char* const Kb = static_cast<const unsigned char*>(a.K) + chunk0 * 16 + row0 * a.k_tok;
    const unsigned char* const Vb = static_cast<const unsigned char*>(a.V) + chunk0 * 16 + row0 * a.v_tok;
    TileCursor ld = seg;
    int ld_left = static_cast<int>(w1 - w0);   // tiles that have not been asked for
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
      Kh = Kb + kv * a.k_head;
      Vh = Vb + kv * a.v_head;
    };
    const uint64_t policy = read_once();
    const uint32_t lane_c = turn<kRow>(row0, chunk0);
    const auto copy_to = [&](uint32_t dst, int j) { return dst + (lane_c ^ ((j * kRows & 7) << 4)) + j * kRows * kRow; };
    // rows at base + the lane's offset of each (whole: of each 16)
    const auto copy_rows = [&](uint32_t dst, const unsigned char* base, int64_t off, int64_t tok) {
      if (whole) {
        const int64_t step = tok * kRows;
#pragma unroll
        for (int m = 0; m < kSub; ++m) {
          const unsigned char* src = base + (kSub == 1 ? off : __shfl_sync(~0u, off, 16 * m));
          constexpr int kEach = kCopies / kSub;
          if (live == kAll) {
#pragma unroll
            for (int j = 0; j < kEach; ++j, src += step) copy16(copy_to(dst, m * kEach + j), src, policy);
          } else {
#pragma unroll
            for (int j = 0; j < kEach; ++j, src += step)
              copy16(copy_to(dst, m * kEach + j), src, policy, (live >> (m * 16 + j * kRows + row0)) & 1);
          }
        }
      } else {
        const unsigned char* const first = base - row0 * tok;
#pragma unroll
        for (int j = 0; j < kCopies; ++j) {
          const int row = j * kRows + row0;
          const int64_t at = __shfl_sync(~0u, off, row);
          const bool on = (live >> row) & 1;
          copy16(copy_to(dst, j), on ? first + at : first, policy, on);
        }
      }
    };
    // K, then V, of the tile at ld go to a slot; the two calls of a tile stand around the products of another
    const auto issue_k = [&](int slot) {
      if (ld_left > 0) {
        const bool ok = static_cast<uint32_t>(id) < static_cast<uint32_t>(a.n_pages);
        live = mask & __ballot_sync(~0u, ok);
        if (!ok) id = in_page = 0;
        if (lane == 0) {
          masks[slot] = live;
          if (live != mask) *a.status = HHR_ERR_BAD_INDEX;
        }
        copy_rows(ring + slot * 2 * kTile, Kh, id * a.k_page + in_page * a.k_tok, a.k_tok);
      }
      copy_commit();
    };
    const auto issue_v = [&](int slot) {
      if (ld_left > 0) {
        copy_rows(ring + slot * 2 * kTile + kTile, Vh, id * a.v_page + in_page * a.v_tok, a.v_tok);
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
    const uint32_t lane_k = turn<kRow>(lane & 15, lane >> 4);
    const uint32_t lane_v = turn<kRow>((lane & 7) + (lane >> 4) * 8, (lane >> 3) & 1);
    int slot = 0;
    int64_t f = w0;

    while (true) {   // units of this warp's range
      const int g_kv = seg.u / a.chunks, first_head = (seg.u - g_kv * a.chunks) * a.chunk;
      const int heads = min(a.chunk, a.r - first_head);
      const int head0 = g_kv * a.r + first_head;
      const UnitSpan span(seg, f, w1);
      int left = span.left;

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
              qf[k][n][0] = on ? x.x ^ a.flip : 0;
              qf[k][n][1] = on ? x.y ^ a.flip : 0;
            } else {
              const uint32_t x = *reinterpret_cast<const uint32_t*>(row + k * 16 + 2 * t4);
              const uint32_t y = *reinterpret_cast<const uint32_t*>(row + k * 16 + 8 + 2 * t4);
              qf[k][n][0] = on ? x ^ a.flip : 0;
              qf[k][n][1] = on ? y ^ a.flip : 0;
            }
          }
        } else {   // bf16 queries of an 8-bit cache
          float top = 0;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint2 x = *reinterpret_cast<const uint2*>(row + k * 16 + 4 * t4);
            qf[k][n][0] = on ? x.x ^ a.flip : 0;
            qf[k][n][1] = on ? x.y ^ a.flip : 0;
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
          m[n][e] = -INFINITY;        // the largest product so far
          base[n][e] = l[n][e] = 0;   // m, or 0 while there is none: products of -inf weigh nothing
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
            ldsm4(r, kt + chunk_at<kRow>(lane_k, S::kE4 ? k : 2 * k) + i * 16 * kRow);
            if constexpr (S::kE4) {
              uint32_t x[4], y[4];
              widen(r[0], x[0], x[2]);
              widen(r[1], x[1], x[3]);
              widen(r[2], y[0], y[2]);
              widen(r[3], y[1], y[3]);
              dot(i, k, x);
              dot(i, k + 1, y);
            } else {
              dot(i, k, r);
            }
          }
        __syncwarp();
        issue_k(slot);
        // weights: lane (g, t4) holds tokens g and g + 8 of heads 2 t4 and 2 t4 + 1
        const bool some = rows != kAll;
        bool grown = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < kSub; ++i) {
            float(&x)[4] = s[i][0][n];
            if constexpr (kSums == 2) {
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] += s[i][kSums - 1][n][e];
            }
            if (some) {
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
              if (top > m[n][e]) {   // the same for the 8 lanes of a column
                const float by = m[n][e] == -INFINITY ? 1.0f : ex2((m[n][e] - top) * sc[n][e]);
                m[n][e] = base[n][e] = top;
                l[n][e] *= by;
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                  o[n][j][e] *= by;
                  o[n][j][e + 2] *= by;
                }
              }
            }
        }
        uint32_t p[kSub][NT][2][kTerms];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < kSub; ++i) {
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = ex2(fmaf(s[i][0][n][e] - base[n][e & 1], sc[n][e & 1], kLift));
            if (some) {   // (a scale of zero makes them numbers)
              if (!((rows >> (16 * i + g)) & 1)) w[0] = w[1] = 0;
              if (!((rows >> (16 * i + g + 8)) & 1)) w[2] = w[3] = 0;
            }
            l[n][0] += w[0] + w[2];
            l[n][1] += w[1] + w[3];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              split<TM>(w[2 * e], w[2 * e + 1], p[i][n][e]);
#pragma unroll
              for (int k = 0; k < kTerms; ++k) p[i][n][e][k] = transposed(p[i][n][e][k]);
            }
          }
        copy_wait<kLead>();
        __syncwarp();
        // O^T += V^T P^T, the tile's product a sum of its own
        constexpr int kStep = S::kE4 ? 2 : 1;   // 16-column products of a load
#pragma unroll
        for (int j = 0; j < D / 16; j += kStep) {
          float t[kStep][NT][4];
#pragma unroll
          for (int h = 0; h < kStep; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) t[h][n][e] = 0;
#pragma unroll
          for (int i = 0; i < kSub; ++i) {
            const auto add = [&](int h, const uint32_t (&r)[4]) {
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int k = kTerms - 1; k >= 0; --k) mma<TM>(t[h][n], r, p[i][n][0][k], p[i][n][1][k]);
            };
            uint32_t r[4];
            if constexpr (S::kE4) {
              // a transposed 2-byte element is columns 2 g and 2 g + 1 of a token: rows g and g + 8 of the product
              ldsm4_trans(r, vt + chunk_at<kRow>(lane_k, j) + i * 16 * kRow);
#pragma unroll
              for (int e = 0; e < 4; ++e) r[e] = __byte_perm(r[e], 0, 0x3120);
              uint32_t x[4], y[4];
              widen(r[0], x[0], x[1]);
              widen(r[1], x[2], x[3]);
              widen(r[2], y[0], y[1]);
              widen(r[3], y[2], y[3]);
              add(0, x);
              add(1, y);
            } else {
              ldsm4_trans(r, vt + chunk_at<kRow>(lane_v, 2 * j) + i * 16 * kRow);
              add(0, r);
            }
          }
#pragma unroll
          for (int h = 0; h < kStep; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[n][j + h][e] += t[h][n][e];
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
      if (span.began && span.ends) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int h = n * 8 + 2 * t4 + e;
            if (h >= heads) continue;
            const float inv = paged_inverse(l[n][e], a.v_scale);
            const size_t row = static_cast<size_t>(seg.b) * a.Hq + head0 + h;
            if (a.lse && g == 0) a.lse[row] = paged_log_sum(paged_quarter(m[n][e], sc[n][e]), l[n][e], kLift);
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
            if (g == 0) *reinterpret_cast<float2*>(row + D) = make_float2(paged_quarter(m[n][e], sc[n][e]), l[n][e]);
          }
        if (lane == 0) s_open[2 * warp + last] = {span.x0, span.x1, seg.b, seg.u};
      }
      if (f == w1) break;
      seg.at = seg.t.end - 1;
      seg.next<kTokens>(a, units);
    }
  }
  __syncthreads();

  // ---- open states, in the order of the tokens: those of one unit are joined.  They lie over the rings of adjacent
  // warps, but for that of a warp that went on to another unit.
  float* const rings = reinterpret_cast<float*>(smem + S::kRing);
  if (warp == 0) {   // a lane per state lists the joins
    int64_t x0 = 0, x1 = 0;
    if (lane < 2 * kWarps) {
      x0 = s_open[lane].x0;
      x1 = s_open[lane].x1;
    }
    const uint32_t open = __ballot_sync(~0u, x1 != 0);
    const uint32_t ahead = open & ((1u << lane) - 1);
    const int64_t x0_ahead = __shfl_sync(~0u, x0, ahead ? 31 - __clz(ahead) : 0);
    const bool begins = x1 != 0 && (!ahead || x0_ahead != x0);   // the first state of its unit
    const uint32_t all = __ballot_sync(~0u, begins);
    if (lane == 0) {
      s_joins = min(__popc(all), kWarps + 1);
      s_side[0] = s_side[1] = -1;
    }
    __syncwarp();
    const int k = __popc(all & ((1u << lane) - 1));
    if (begins && k <= kWarps) {   // (more units than that: lengths that changed during the call)
      const uint32_t behind = all & ~((2u << lane) - 1);
      const uint32_t upto = open & (behind ? (1u << (__ffs(behind) - 1)) - 1 : ~0u);
      const int i1 = 31 - __clz(upto), wa = lane >> 1, wb = i1 >> 1;
      const int b = s_open[lane].b, u = s_open[lane].u;
      const int g_kv = u / a.chunks, first_head = (u - g_kv * a.chunks) * a.chunk;
      const bool inside = x0 >= f0 && x1 <= f1;
      const int side = x0 >= f0;
      Join& j = s_join[k];
      j.base = rings + wa * (S::kRingWarp / 4);
      j.last = (i1 & 1) ? nullptr : a.firsts + static_cast<size_t>(c * kWarps + wb) * a.state;
      j.to = inside ? nullptr : a.parts + static_cast<size_t>(2 * c + side) * a.state;
      j.out_row = static_cast<size_t>(b) * a.Hq + g_kv * a.r + first_head;
      j.x0 = x0;
      j.x1 = x1;
      j.stride = S::kRingWarp / 4;
      j.n = wb - wa + 1;
      j.heads = min(a.chunk, a.r - first_head);
      if (!inside) s_side[side] = k;
    }
  }
  __syncthreads();
  join_states<TQ, TM, D, kThreads>(a, s_join, s_joins);

  if (s_side[0] >= 0 || s_side[1] >= 0) {
    // Units shared with CTAs before (0) and behind (1).  The last of a unit's CTAs to arrive joins their states from L2.
    // (The barrier and the acquire-release addition order every thread's state before the addition and the other CTAs'
    // states behind it.)
    __syncthreads();
    if (lane == 0 && warp < 2) {
      const int k = s_side[warp];
      int n = 0;
      if (k >= 0) {
        Join& j = s_join[k];
        const int c0 = deal.cta_of(j.x0, gridDim.x);
        n = max(1, deal.cta_of(j.x1 - 1, gridDim.x) - c0 + 1);
        uint32_t* const count = a.counters + c0;
        uint32_t old;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(count) : "memory");
        if (old == static_cast<uint32_t>(n - 1)) {
          *count = 0;
          // the states of the CTAs behind the first, and the first one's
          j.base = a.parts + static_cast<size_t>(2 * (c0 + 1)) * a.state;
          j.last = a.parts + static_cast<size_t>(2 * c0 + 1) * a.state;
          j.to = nullptr;
          j.stride = 2 * a.state;
          j.n = n;
        } else {
          n = 0;
        }
      }
      s_last[warp] = n;
    }
    __syncthreads();
#pragma unroll 1
    for (int side = 0; side < 2; ++side)
      if (s_last[side]) join_states<TQ, TM, D, kThreads>(a, s_join + s_side[side], 1);
  }

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

}

// Launches the variant for D and the heads of a unit.
template <typename TQ, typename TC, int D, int NT, bool kFine>
cudaError_t launch_paged_kernel(const PagedArgs& a, int grid, cudaStream_t s) {
  using S = PagedShape<TQ, TC, D, NT>;
  static std::atomic<size_t> raised[kMaxDevices];
  const auto kern = paged_kernel<TQ, TC, D, NT, kFine>;
  if (cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), S::kSmem, raised)) return e;
  return launch_dependent<PagedArgs>(kern, dim3(grid), S::kThreads, S::kSmem, s, a);
}

// Most heads of a unit, by the registers of its sums: D / 16 x 4 floats a lane for 8 heads.
inline int paged_max_heads(int d) { return d == 64 ? 32 : d == 128 ? 24 : 16; }

template <typename TQ, typename TC, int D, int NT>
cudaError_t launch_paged_out(const PagedArgs& a, int grid, cudaStream_t s) {
  if constexpr (std::is_same<TC, __nv_bfloat16>::value)
    if (a.out_f32) return launch_paged_kernel<TQ, TC, D, NT, true>(a, grid, s);
  return launch_paged_kernel<TQ, TC, D, NT, false>(a, grid, s);
}

template <typename TQ, typename TC>
cudaError_t launch_paged_typed(const PagedArgs& a, int d, int grid, cudaStream_t s) {
  const int nt = (a.chunk + 7) / 8;
  if (d == 64) {
    if (nt == 1) return launch_paged_out<TQ, TC, 64, 1>(a, grid, s);
    if (nt == 2) return launch_paged_out<TQ, TC, 64, 2>(a, grid, s);
    if (nt == 3) return launch_paged_out<TQ, TC, 64, 3>(a, grid, s);
    return launch_paged_out<TQ, TC, 64, 4>(a, grid, s);
  }
  if (d == 128) {
    if (nt == 1) return launch_paged_out<TQ, TC, 128, 1>(a, grid, s);
    if (nt == 2) return launch_paged_out<TQ, TC, 128, 2>(a, grid, s);
    return launch_paged_out<TQ, TC, 128, 3>(a, grid, s);
  }
  if (nt == 1) return launch_paged_out<TQ, TC, 256, 1>(a, grid, s);
  return launch_paged_out<TQ, TC, 256, 2>(a, grid, s);
}

// One translation unit per pair of types (paged_*.cu).
cudaError_t launch_paged_bf16(const PagedArgs& a, int d, int grid, cudaStream_t s);
cudaError_t launch_paged_f16(const PagedArgs& a, int d, int grid, cudaStream_t s);
cudaError_t launch_paged_bf16_e4m3(const PagedArgs& a, int d, int grid, cudaStream_t s);
cudaError_t launch_paged_f16_e4m3(const PagedArgs& a, int d, int grid, cudaStream_t s);

}  // namespace hhr
