"""Every entry point with a default workspace under graph capture: the memory
is the graph's own, so that graphs captured on one stream can be replayed at
once, beside eager calls on that stream."""
import weakref

import pytest
import torch

from tests.standins import Gpus, Stream, calls
from tests.test_quantized_serving_step import BF, DEV, Step, run, same, sv

TAKE_WORKSPACE = ("verify", "sparse", "static", "head_quantized", "logprobs")


def scratch(gpus):
    """Workspaces that the calls allocated so far."""
    return [t for t in gpus.made if t.dtype == torch.uint8 and t.numel() >= gpus.need]


@pytest.mark.parametrize("name", TAKE_WORKSPACE)
def test_captured_calls_own_their_workspace(monkeypatch, name):
    gpus = Gpus(monkeypatch)
    monkeypatch.setattr(sv(), "_default_ws", {})
    side = Stream(0)
    with gpus.stream(side):
        gpus.captured.append(side)
        calls()[name]()
        calls()[name]()
        gpus.captured.clear()
        captured = scratch(gpus)
        assert len(captured) == 2 and sv()._default_ws == {}
        calls()[name]()
        calls()[name]()
        eager = scratch(gpus)[2:]
        assert len(eager) == 1                     # kept between eager calls
        gpus.captured.append(side)
        calls()[name]()
        assert len(scratch(gpus)) == 4             # and not given to a later captured one


@pytest.mark.gpu
def test_whole_steps_replayed_at_once():
    """Two steps (quantised head, static head, verify, log-probabilities of long rows) captured on one stream with
    default workspaces, replayed on two streams while an eager step runs on the stream they were captured on."""
    steps = [Step(20 + i, V=70000) for i in range(3)]
    weights = [sv().spec_quantize_rows(s.W) for s in steps]

    def whole(i):
        s = steps[i]
        head = sv().spec_draft_head_static(s.h, s.W, s.ids, s.cs, dtype=BF)
        return run(s, *weights[i]) + [head]
    want = [whole(i) for i in range(3)]
    torch.cuda.synchronize()
    side, a, b = (torch.cuda.Stream() for _ in range(3))
    with torch.cuda.stream(side):
        whole(0)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(whole(i))
        graphs.append(g)
    for _ in range(6):
        for o in outs:
            for v in o:
                v.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(a):
            graphs[0].replay()
        with torch.cuda.stream(b):
            graphs[1].replay()
        with torch.cuda.stream(side):
            eager = whole(2)
        torch.cuda.synchronize()
        assert same(outs[0], want[0]) and same(outs[1], want[1]) and same(eager, want[2])


def test_a_workspace_keeps_the_buffers_that_graphs_use(monkeypatch):
    gpus = Gpus(monkeypatch)
    side = Stream(0)
    ws = sv().Workspace(torch.device("cuda", 0))
    first = weakref.ref(ws.get(1000))
    gpus.made.clear()
    ws.get(2000)
    assert first() is None                         # replaced, and no graph uses it
    with gpus.stream(side):
        gpus.captured.append(side)
        for _ in range(3):
            used = weakref.ref(ws.get(1500))
        gpus.captured.clear()
    ws.get(1 << 20)
    gpus.made.clear()
    assert used() is not None and ws.buf is not used() and ws.buf.numel() == 1 << 20
    del ws
    assert used() is None


@pytest.mark.gpu
def test_a_workspace_that_grows_after_a_capture():
    """A larger eager call replaces the buffer of a captured one; tensors made since keep their values through replays."""
    g = torch.Generator().manual_seed(41)
    x = torch.randn(50, 70000, generator=g).to(BF).to(DEV)
    big = torch.randn(400, 70000, generator=g).to(BF).to(DEV)
    t = torch.randint(0, 70000, (400,), generator=g).to(torch.int32).to(DEV)
    ws = sv().Workspace(DEV)
    want = sv().spec_token_logprobs(x, t[:50], 9, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = sv().spec_token_logprobs(x, t[:50], 9, workspace=ws)
    size = ws.buf.numel()
    ref = sv().spec_token_logprobs(big, t, 9, workspace=ws)
    assert ws.buf.numel() > size
    others = [torch.full((size,), 7, dtype=torch.uint8, device=DEV) for _ in range(4)]
    for _ in range(4):
        for v in out:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, want)
        assert all((o == 7).all() for o in others)
        assert same(sv().spec_token_logprobs(big, t, 9, workspace=ws), ref)
