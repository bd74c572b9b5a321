"""Two host threads on one stream: the launches of their calls may alternate
there, so their default workspaces are apart."""
import threading

import pytest
import torch

from tests.standins import Gpus, calls
from tests.test_quantized_serving_step import BF, DEV, same, sv


def at_once(*fs):
    """Runs each of fs in a thread of its own, all alive to the end; their results."""
    barrier, got = threading.Barrier(len(fs)), [None] * len(fs)

    def body(i):
        barrier.wait()
        try:
            got[i] = fs[i]()
        finally:
            barrier.wait()
    threads = [threading.Thread(target=body, args=(i,)) for i in range(len(fs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return got


@pytest.mark.parametrize("name", ("verify", "sparse", "static", "head_quantized", "logprobs"))
def test_threads_have_default_workspaces_of_their_own(monkeypatch, name):
    gpus = Gpus(monkeypatch)
    monkeypatch.setattr(sv(), "_default_ws", {})

    def buffers():
        calls()[name]()
        calls()[name]()
    at_once(buffers, buffers)
    assert len([t for t in gpus.made if t.dtype == torch.uint8 and t.numel() >= gpus.need]) == 2


@pytest.mark.gpu
def test_threads_on_one_stream():
    """Calls of several launches from four threads on the current stream, against the same calls one by one."""
    g = torch.Generator().manual_seed(31)
    xs = [(torch.randn(40, 70000 + 512 * i, generator=g) * 3).to(BF).to(DEV) for i in range(2)]
    toks = [torch.randint(0, 70000, (40,), generator=g).to(torch.int32).to(DEV) for _ in range(2)]
    hs = [torch.randn(40, 2048, generator=g).to(BF).to(DEV) for _ in range(2)]
    W = sv().spec_quantize_rows((torch.randn(600, 2048, generator=g) / 45).to(BF).to(DEV))
    ids = torch.arange(600, dtype=torch.int32, device=DEV)
    fs = [lambda x=x, t=t: sv().spec_token_logprobs(x, t, 8) for x, t in zip(xs, toks)]
    fs += [lambda h=h: [sv().spec_draft_head_quantized(h, *W, ids, 1)] for h in hs]
    want = [f() for f in fs]
    torch.cuda.synchronize()
    got = at_once(*[lambda f=f: [f() for _ in range(50)] for f in fs])
    torch.cuda.synchronize()
    for w, many in zip(want, got):
        assert all(same(w, one) for one in many)
