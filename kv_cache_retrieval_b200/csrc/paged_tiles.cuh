// Which tiles a warp of hhr_paged_attend has: the arguments of its kernel, a sequence's tiles, the walk over them, and the
// even deal of the call's tiles over the card's warps.  Plain arithmetic, the same on the host (its tests run there).
//
// Lengths are read more than once.  They must not change during a call; if they do all the same, the answers are wrong but
// every walk here still ends and every index stays in its range: a cursor always stands on a tile (of rows that are no
// tokens, if its sequence has none left), and the CTAs that share a unit are CTAs of the grid.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace hhr {

#define PAGED_BOTH __host__ __device__ __forceinline__

constexpr int kPagedMaxGrid = 160;   // CTAs that take part in a call (one per SM)
constexpr int kPagedMaxWarps = 12;   // warps of a CTA

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
  float* firsts;               // [kPagedMaxGrid][kPagedMaxWarps]: states of the units that a warp ends and did not begin
  int64_t q_seq;                                              // elements
  int64_t k_page, k_head, k_tok, v_page, v_head, v_tok;       // bytes
  float scale_log2, v_scale;   // |scale| k_scale log2(e)
  uint32_t flip;               // the signs of two 16-bit values if the scale is negative: the queries take it
  int B, Hq, Hkv, page, n_pages, table_cols, table_stride, window, out_f32;
  int r, chunk, chunks;        // query heads of a KV head, of a unit (at most 8 NT), and units of a KV head
  int state;                   // floats of a state
  uint32_t page_magic;         // n / page = (umulhi(n, magic) + n) >> shift for n < 2^31
  int page_shift;
  int min_tiles;               // a warp takes at least that many
};

// Tiles of a sequence: [first, end).
struct TileRange {
  int lo, len, first, end;
};

template <int kTokens>
PAGED_BOTH TileRange tile_range(const PagedArgs& a, int b) {
  TileRange t;
  t.len = a.lens[b];
  if (t.len < 0 || t.len > a.table_cols * a.page) t.len = 0;
  t.lo = a.window && t.len > a.window ? t.len - a.window : 0;
  t.first = t.lo / kTokens;
  t.end = static_cast<int>((static_cast<uint32_t>(t.len) + (kTokens - 1)) / kTokens);
  return t;
}

// A tile of the call: sequence, unit of the sequence, tile of the unit.
struct TileCursor {
  TileRange t;
  int b, u, at;

  // On the unit's tile that stands `off` tiles of the call behind sequence b's first one; t is that sequence's.
  PAGED_BOTH void place(int64_t off, int units) {
    stand();
    const int n = t.end - t.first;
    const int64_t last = static_cast<int64_t>(n) * units - 1;
    off = off < 0 ? 0 : off > last ? last : off;
    u = static_cast<int>(static_cast<uint64_t>(off) >> 32 ? off / n : static_cast<uint32_t>(off) / static_cast<uint32_t>(n));
    at = t.first + static_cast<int>(off - static_cast<int64_t>(u) * n);
  }
  template <int kTokens>
  PAGED_BOTH void next(const PagedArgs& a, int units) {   // the next tile has to exist
    if (++at < t.end) return;
    if (++u == units) {
      u = 0;
      while (b + 1 < a.B) {
        t = tile_range<kTokens>(a, ++b);
        if (t.first < t.end) break;
      }
      stand();
    }
    at = t.first;
  }
  PAGED_BOTH void stand() {   // (a sequence without tiles: its length changed since the tiles were dealt out)
    if (t.end <= t.first) t.end = t.first + 1;
  }
};

// What a warp that is at tile f of the call, where `seg` stands, and whose tiles end at w1 has of seg's unit.
struct UnitSpan {
  int64_t x0, x1;      // the unit's tiles
  int left;            // tiles of it to go, at least 1
  bool began, ends;    // whether the warp has the unit's first and last one
  PAGED_BOTH UnitSpan(const TileCursor& seg, int64_t f, int64_t w1) {
    x0 = f - (seg.at - seg.t.first);
    x1 = x0 + (seg.t.end - seg.t.first);
    began = f == x0;
    ends = x1 <= w1;
    left = static_cast<int>((ends ? x1 : w1) - f);
  }
};

// The deal of `total` tiles (fewer than 2^36) over n_active warps each of n_warps / n_active CTAs.
struct TileDeal {
  int64_t total, quot;
  uint32_t n_warps, rem;
  int n_active;
  PAGED_BOTH TileDeal(int64_t tiles, int ctas, int warps) {
    total = tiles;
    n_active = warps;
    n_warps = static_cast<uint32_t>(ctas) * warps;
    quot = total >> 32 ? total / n_warps : static_cast<int64_t>(static_cast<uint32_t>(total) / n_warps);
    rem = static_cast<uint32_t>(total - quot * n_warps);
  }
  // Warp i of them takes [first_of(i), first_of(i + 1)).
  PAGED_BOTH int64_t first_of(uint32_t i) const {
    i = i < n_warps ? i : n_warps;
    return quot * i + rem * i / n_warps;
  }
  // The CTA of the warp whose range holds tile x, the last with total * i / n_warps <= x; one of the grid for any x.
  PAGED_BOTH int cta_of(int64_t x, int grid) const {
    const uint64_t c = (static_cast<uint64_t>(x + 1) * n_warps - 1) / static_cast<uint64_t>(total > 0 ? total : 1) / n_active;
    return c < static_cast<uint64_t>(grid) ? static_cast<int>(c) : grid - 1;
  }
};

}  // namespace hhr
