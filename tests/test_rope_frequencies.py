"""YaRN's frequencies where the ramp's end lies beyond the last pair.

The published ramp runs over the pair index from lo = max(floor(dim(high)), 0) to hi = min(ceil(dim(low)), rot - 1), with
dim(t) = rot ln(orig / (2 pi t)) / (2 ln base), the (real) index of the pair that makes t turns over orig tokens.  rot - 1
lies beyond the last pair, rot/2 - 1: where the slowest pair still makes more than a turn, hi is beyond the last pair and
the ramp does not reach 1 within them."""
import math

import pytest
import torch

import kv_cache_retrieval_b200 as hhr
from kv_cache_retrieval_b200 import build as kbuild


@pytest.fixture(scope="module", autouse=True)
def built():
    kbuild.build()


# rot, base, factor, orig, hi: worked out by hand from the formula above
@pytest.mark.parametrize("rot,base,factor,orig,hi", [
    (128, 1e4, 4.0, 65536, 65), (128, 1e4, 8.0, 131072, 70), (32, 1e4, 4.0, 65536, 17), (16, 1e4, 4.0, 32768, 8),
    (4, 5e5, 4.0, 32768, 2), (4, 1e4, 4.0, 2 ** 31 - 1, 3), (128, 5e5, 4.0, 32768, 42), (64, 1e6, 4.0, 32768, 20)])
def test_yarn_ramp_reaches_its_published_end(rot, base, factor, orig, hi):
    turns = lambda t: rot * math.log(orig / (2 * math.pi * t)) / (2 * math.log(base))  # noqa: E731
    assert hi == min(math.ceil(turns(1.0)), rot - 1)
    lo = max(math.floor(turns(32.0)), 0)
    f, _ = hhr.rope_freqs(rot, base=base, scaling="yarn", factor=factor, orig=orig, device="cpu")
    j = torch.arange(rot // 2, dtype=torch.float64)
    plain = base ** (-2 * j / rot)
    width = max(hi - lo, 0.001)
    s = ((j - lo) / width).clamp(0, 1)
    assert torch.allclose(f, plain * (1 - s) + plain / factor * s, rtol=1e-13, atol=0)
    # the share of the stretch that the last pair has, read back from its frequency
    last = (1 - f[-1] / plain[-1]) / (1 - 1 / factor)
    assert float(last) == pytest.approx(min(1.0, max(0.0, (rot // 2 - 1 - lo) / width)), abs=1e-12)
