"""The deal of the paged attention's tiles over the card's warps (csrc/paged_tiles.cuh), compiled for the host: every tile
has one warp, and walks end within their tiles even if lengths change under a call."""
import ctypes as C
import os
import random
import subprocess

import pytest

from kv_cache_retrieval_b200 import build as kbuild

SOURCE = r"""
#include <cmath>
#include <cstdlib>
#include <vector>
#include "paged_tiles.cuh"
using namespace hhr;
constexpr int kTokens = 16;

// Walks all warps as the kernel does: begins at its first tile, unit by unit, and a second cursor tile by tile.  change:
// lengths are drawn anew at every step, after the tiles were dealt out.  seen[tile of (b, u)]: how often a warp had it.
// Returns 0, or where it went wrong.
extern "C" int walk(int32_t* lens, int B, int units, int window, int cols, int page, int ctas, int warps, int change,
                    unsigned seed, int32_t* seen, int seen_stride) {
  PagedArgs a = {};
  a.lens = lens;
  a.B = B;
  a.window = window;
  a.table_cols = cols;
  a.page = page;
  std::vector<int64_t> before(B + 1, 0);
  for (int b = 0; b < B; ++b) {
    const TileRange t = tile_range<kTokens>(a, b);
    before[b + 1] = before[b] + (t.end - t.first);
  }
  const int64_t total = before[B] * units;
  if (total == 0) return 0;
  srand(seed);
  const auto shake = [&] {
    if (change)
      for (int b = 0; b < B; ++b) lens[b] = rand() % 4 == 0 ? rand() % (cols * page + 1) : rand() % 4 == 0 ? -1 : 0;
  };
  const TileDeal deal(total, ctas, warps);
  if (deal.first_of(0) != 0 || deal.first_of(ctas * warps) != total) return 1;
  for (int i = 0; i < ctas * warps; ++i) {
    const int64_t w0 = deal.first_of(i), w1 = deal.first_of(i + 1);
    if (w0 > w1) return 2;
    if (w0 == w1) continue;
    if (!change && (deal.cta_of(w0, ctas) != i / warps || deal.cta_of(w1 - 1, ctas) != i / warps)) return 3;
    TileCursor seg = {};
    seg.b = 0;
    while (seg.b + 1 < B && before[seg.b + 1] * units <= w0) ++seg.b;
    int64_t pre = before[seg.b];
    shake();
    for (;; ++seg.b) {
      seg.t = tile_range<kTokens>(a, seg.b);
      const int n = seg.t.end > seg.t.first ? seg.t.end - seg.t.first : 0;
      if (w0 < (pre + n) * units || seg.b + 1 >= B) break;
      pre += n;
    }
    seg.place(w0 - pre * units, units);
    TileCursor ld = seg;
    for (int64_t k = w0; k < w1; ++k) {   // the loads' cursor
      if (ld.b < 0 || ld.b >= B || ld.u < 0 || ld.u >= units || ld.at < ld.t.first || ld.at >= ld.t.end) return 4;
      if (!change) ++seen[static_cast<size_t>(ld.b * units + ld.u) * seen_stride + ld.at];
      shake();
      if (k + 1 < w1) ld.next<kTokens>(a, units);
    }
    int64_t f = w0;
    for (int64_t step = 0;; ++step) {
      if (step > w1 - w0) return 5;       // a unit has at least a tile
      const UnitSpan s(seg, f, w1);
      if (s.left < 1 || f + s.left > w1) return 6;
      const int c0 = deal.cta_of(s.x0, ctas), c1 = deal.cta_of(s.x1 - 1, ctas);
      if (c0 < 0 || c0 >= ctas || c1 < 0 || c1 >= ctas) return 7;
      if (!change && (c0 > i / warps || c1 < i / warps || s.x0 > f || s.x1 < f + s.left)) return 8;
      f += s.left;
      if (f == w1) break;
      shake();
      seg.at = seg.t.end - 1;
      seg.next<kTokens>(a, units);
    }
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    at = tmp_path_factory.mktemp("tiles")
    src, lib = at / "tiles.cpp", at / "tiles.so"
    src.write_text(SOURCE)
    cuda = os.path.dirname(os.path.dirname(kbuild._nvcc())) or "/usr/local/cuda"
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-static-libubsan",
                    "-shared", "-fPIC", "-I", kbuild.CSRC, "-I", kbuild.INCLUDE, "-I", os.path.join(cuda, "include"),
                    str(src), "-o", str(lib)], check=True)
    return C.CDLL(str(lib)).walk


def cases(n):
    rng = random.Random(1)
    for _ in range(n):
        B, units = rng.choice([1, 2, 7, 31, 60]), rng.choice([1, 2, 3, 8])
        page, cols = rng.choice([(16, 8), (5, 30), (1, 77), (64, 40)])
        lens = [rng.choice([0, 1, 16, 17, -1, page * cols, page * cols + 1, rng.randint(0, page * cols)]) for _ in range(B)]
        window = rng.choice([0, 0, 1, 16, 100])
        tiles = []
        for n in lens:
            n = n if 0 <= n <= page * cols else 0
            lo = max(0, n - window) if window else 0
            tiles.append((lo // 16, -(-n // 16)) if n else (0, 0))
        total = sum(e - s for s, e in tiles) * units
        ctas = rng.choice([1, 2, 7, 148])
        warps = rng.choice([1, 3, 8, 12])
        while ctas * warps > max(1, total):      # a tile at least for each warp, as the kernel deals them
            ctas, warps = max(1, ctas // 2), max(1, warps // 2)
        yield B, units, page, cols, lens, window, tiles, ctas, warps


def test_every_tile_has_one_warp(walk):
    for B, units, page, cols, lens, window, tiles, ctas, warps in cases(300):
        stride = page * cols // 16 + 2
        seen = (C.c_int32 * (B * units * stride))()
        assert walk((C.c_int32 * B)(*lens), B, units, window, cols, page, ctas, warps, 0, 0, seen, stride) == 0
        for b, (s, e) in enumerate(tiles):
            for u in range(units):
                at = (b * units + u) * stride
                assert list(seen[at:at + stride]) == [int(s <= i < e) for i in range(stride)]


def test_walks_end_when_lengths_change_under_them(walk):
    for i, (B, units, page, cols, lens, window, _, ctas, warps) in enumerate(cases(600)):
        assert walk((C.c_int32 * B)(*lens), B, units, window, cols, page, ctas, warps, 1, i, None, 0) == 0
