"""Calls of one cache on several streams, and their status."""
import threading

import pytest
import torch

import kv_cache_retrieval_b200 as hhr
from test_paged import built, make  # noqa: F401 - built is a fixture

pytestmark = pytest.mark.gpu


def test_streams_do_not_share_the_default_workspace():
    """Calls that overlap on two streams, each as long as several launches, without a workspace of their own."""
    c, q, t = make(2, 8, 2, 128, 16, 700)
    lens = torch.tensor([11200, 8000], dtype=torch.int32, device="cuda")
    want = c.attend(q, t, lens)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(50):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(c.attend(q, t, lens))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    assert c.status() == hhr.HHR_OK
    assert len({w.data_ptr() for w in c._spaces.values()}) == len(c._spaces) == 3
    assert torch.equal(c.attend(q, t, lens), want) and len(c._spaces) == 3


def test_threads_with_a_stream_each_and_no_workspaces():
    c, q, t = make(2, 8, 2, 64, 16, 60)
    lens = [torch.tensor(n, dtype=torch.int32, device="cuda") for n in ([960, 37], [500, 960], [1, 900], [700, 700])]
    want = [c.attend(q, t, n).clone() for n in lens]
    torch.cuda.synchronize()
    fresh = hhr.HHRPagedCache(q_heads=8, kv_heads=2, page=16, head_dim=64, K=c.K, V=c.V)
    torch.cuda.synchronize()
    got, bad = [[] for _ in lens], []
    go = threading.Barrier(len(lens))

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                go.wait()
                for _ in range(100):
                    got[i].append(fresh.attend(q, t, lens[i]))
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001 - reported by the main thread
            bad.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(lens))]
    [x.start() for x in threads]
    [x.join() for x in threads]
    assert not bad, bad
    assert all(torch.equal(o, want[i]) for i in range(len(lens)) for o in got[i])
    assert len({w.data_ptr() for w in fresh._spaces.values()}) == len(lens)


def test_the_status_of_another_streams_call():
    c, q, t = make(2, 4, 2, 64, 16, 6)
    lens = torch.tensor([96, -1], dtype=torch.int32, device="cuda")
    c.attend(q, t, lens.clamp(min=0))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.attend(q, t, lens)
    torch.cuda.current_stream().wait_stream(side)
    assert c.status() == hhr.HHR_ERR_BAD_INDEX
    assert c.status() == hhr.HHR_OK


def test_a_capture_does_not_make_a_workspace():
    """A captured call keeps to a workspace that is zeros now, not at the graph's replays."""
    c, q, t = make(2, 4, 2, 64, 16, 60)
    lens = torch.tensor([960, 700], dtype=torch.int32, device="cuda")
    want = c.attend(q, t, lens)
    torch.cuda.synchronize()
    graph, capturing = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=capturing):
        out = c.attend(q, t, lens)
    assert len(c._spaces) == 1
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    capturing.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(capturing):
        again = c.attend(q, t, lens)
    torch.cuda.synchronize()
    assert torch.equal(again, want) and len(c._spaces) == 2
