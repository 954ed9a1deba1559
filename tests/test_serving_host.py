"""The host side of the serving calls, without a GPU: devices, what is kept between calls, sizes that do not fit."""
import contextlib
import sys

import pytest
import torch

import kv_cache_retrieval_b200 as hhr
from kv_cache_retrieval_b200 import _binding, build as kbuild
from test_paged import attend, desc


@pytest.fixture(scope="module", autouse=True)
def built():
    kbuild.build()


def test_the_retrieval_caches_append_stays_on_its_device(monkeypatch):
    """Both halves of the append, the store and the encoding, run with the cache's device current."""
    c = hhr.HHRCache(batch=1, q_heads=4, kv_heads=2, capacity=64, P=2, k=8, device="cpu")
    current, seen = ["cuda:0"], []

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], str(d)
        yield
        current[0] = before

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(hhr.HHRPagedCache, "append", lambda self, *a, **k: seen.append(("append", current[0])))
    monkeypatch.setattr(_binding, "hhr_encode_keys", lambda *a, **k: seen.append(("encode", current[0])))
    k = torch.zeros(1, 3, 2, 128, dtype=torch.bfloat16)
    c.append(k, k, 0)
    assert seen == [("append", "cpu"), ("encode", "cpu")] and current == ["cuda:0"]


@pytest.mark.parametrize("make", [torch.tensor, lambda x: torch.tensor([x], dtype=torch.float64)])
def test_a_scale_that_changes_in_place_is_read_again(make):
    """Rotations are kept by their values, not by the object that held one."""
    from kv_cache_retrieval_b200.rope import rotation
    m = make(1.25)
    assert rotation(64, 0, m)._obj.mscale == 1.25
    m.fill_(0.5)
    assert rotation(64, 0, m)._obj.mscale == 0.5
    assert rotation(64, 0, 0.5) is rotation(64, 0, m)


@pytest.mark.parametrize("kw,scale", [
    (dict(), 3e38), (dict(), -3e38), (dict(kv_type=3, k_scale=2.0), 2e38), (dict(kv_type=3, k_scale=2.0 ** 100), 2.0 ** 28),
    (dict(), float("nan")), (dict(), -float("inf"))])
def test_scales_beyond_float32_are_refused(kw, scale):
    """The logits are taken in powers of two, scale * k_scale * log2 e: infinite, it would make 0 * inf of the largest."""
    assert attend(desc(**kw), scale=scale) == hhr.HHR_ERR_INVALID_ARG


def test_sizes_beyond_int32_are_not_cut_off(monkeypatch):
    """The library takes int32; ctypes drops what is beyond.  (Tensors without memory: nothing is called.)"""
    paged, rope = (sys.modules["kv_cache_retrieval_b200." + m] for m in ("paged", "rope"))
    calls = []
    monkeypatch.setattr(paged, "on_device", lambda index, fn, *args: calls.append(args) or 0)
    monkeypatch.setattr(rope, "on_device", lambda index, fn, *args: calls.append(args) or 0)
    c = hhr.HHRPagedCache(q_heads=8, kv_heads=2, pages=4, head_dim=64, device="cpu")
    table, lens = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    q = torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    for window, passed in ((0, 0), (7, 7), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1)):
        c.attend(q, table, lens, window=window)
        assert calls.pop()[8] == passed
    c.attend(q, table, lens, window=-2 ** 32)      # refused by the library
    assert calls.pop()[8] == -1
    many = 2 ** 32 + 3
    k = torch.empty(many, 2, 64, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="2\\^31"):
        c.append(k, k, torch.empty(many, dtype=torch.int32, device="meta"), table)
    with pytest.raises(ValueError, match="2\\^31"):
        c.attend(q, torch.empty(3, many, dtype=torch.int32, device="meta"), lens)
    x = torch.empty(many, 1, 2, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="2\\^31"):
        rope._rotate(x, torch.empty(many, dtype=torch.int32, device="meta"), torch.empty(1, device="meta"), 0, 1.0, x)
    with pytest.raises(ValueError, match="2\\^31"):
        hhr.HHRPagedCache(q_heads=2 ** 32 + 8, kv_heads=2, pages=4, head_dim=64, device="cpu")
    assert not calls


def test_a_cache_can_be_copied():
    import copy
    c = hhr.HHRPagedCache(q_heads=8, kv_heads=2, pages=4, head_dim=64, device="cpu")
    d = copy.deepcopy(c)
    assert d.K.data_ptr() != c.K.data_ptr() and d.desc.Hq == 8
