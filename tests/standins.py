"""Stand-ins for torch's GPU calls and the C library, so that the Python half
of the entry points (who allocates on which stream, which workspace a call
gets, which device is current) is tested without a GPU.

Tensors are CPU tensors that say they are on a GPU.  Each one made through
torch.empty knows the stream that was current (`made_on`) and the streams that
were recorded with it (`recorded`)."""
import contextlib
import itertools

import torch

import speculative_sampling_verification_vocab_amd as sv

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


class Stream:
    handles = itertools.count(0x70000001, 0x10)

    def __init__(self, device, handle=None):
        self.device = torch.device("cuda", device)
        self.cuda_stream = next(Stream.handles) if handle is None else handle

    def __repr__(self):
        return f"<stream {self.cuda_stream:#x} of {self.device}>"


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on GPU `index`."""

    @classmethod
    def of(cls, t, index=0):
        t = torch.Tensor._make_subclass(cls, t)
        t.index, t.recorded, t.made_on = index, [], None
        return t

    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", getattr(self, "index", 0)))

    def record_stream(self, stream):
        self.recorded.append(stream)


class Library:
    """The C library: every call succeeds and is noted with the device that was current."""

    def __init__(self, gpus):
        self.gpus, self.calls = gpus, []

    def __getattr__(self, name):
        if name.endswith("_workspace_bytes"):
            return lambda *a: self.gpus.need
        if name.endswith("_launch_count"):
            return lambda *a: 1

        def call(*args):
            self.calls.append((name, self.gpus.current_device(), args))
            return 0
        return call


class Gpus:
    """Two devices with their current streams; patches torch.cuda, torch.empty and the library."""

    def __init__(self, monkeypatch, need=1 << 12):
        self.default = [Stream(i, 0) for i in range(2)]
        self.at, self.dev = list(self.default), 0
        self.captured, self.made, self.need = [], [], need
        self.lib = Library(self)
        empty = torch.empty

        def make(*size, dtype=None, device=None, **kw):
            if device is None or torch.device(device).type != "cuda":
                return empty(*size, dtype=dtype, device=device, **kw)
            d = torch.device(device).index
            t = OnGpu.of(empty(*size, dtype=dtype), d)
            t.made_on = self.at[d]
            self.made.append(t)
            return t
        monkeypatch.setattr(torch, "empty", make)
        monkeypatch.setattr(torch, "empty_like",
                            lambda t, dtype=None: make(t.shape, dtype=dtype or t.dtype, device=t.device))
        for name in ("current_device", "current_stream", "stream", "device"):
            monkeypatch.setattr(torch.cuda, name, getattr(self, name))
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.at[self.dev] in self.captured)
        monkeypatch.setattr(sv, "_raw_current_stream", lambda index: self.at[index].cuda_stream)
        monkeypatch.setattr(sv._native, "load", lambda: self.lib)

    def current_device(self):
        return self.dev

    def current_stream(self, device=None):
        return self.at[self.dev if device is None else torch.device(device).index]

    @contextlib.contextmanager
    def stream(self, s):
        kept = self.dev, list(self.at)
        self.dev, self.at[s.device.index] = s.device.index, s
        try:
            yield
        finally:
            self.dev, self.at = kept

    @contextlib.contextmanager
    def device(self, d):
        kept, self.dev = self.dev, torch.device(d).index
        try:
            yield
        finally:
            self.dev = kept


def tensor(shape, dtype, index=0):
    t = torch.zeros(shape, dtype=torch.uint8 if dtype in (F8, E8) else dtype)
    return OnGpu.of(t.view(dtype) if dtype in (F8, E8) else t, index)


def calls(index=0):
    """Every entry point that takes a stream: name -> f(**keywords) on small tensors of GPU `index`."""
    def t(shape, dtype):
        return tensor(shape, dtype, index)
    B, K, V, d, P, L = 2, 3, 40, 256, 2, 8
    target, draft = t((B, K + 1, V), BF), t((B, K, V), BF)
    toks, uni, ids = t((B, K), I32), t((B, K + 1, 2), F32), t((4,), I32)
    h, W = t((B, K, d), BF), t((V, d), BF)
    wc, ws = t((V, d), F8), t((V, d // 128), E8)
    codes, scales, staging = t((P, B, L, 128), F8), t((P, B, L, 1), E8), t((P, B, K, 128), BF)
    n, at = t((B,), I32), t((B,), I32)
    cids = t((B, K, 2), I32)
    return {
        "verify": lambda **k: sv.spec_verify(target, draft, toks, uni, return_probs=True, **k),
        "verify_noalloc": lambda **k: sv.spec_verify_noalloc(target, draft, toks, uni,
                                                             out=(t((B,), I32), t((B, K + 1), I32)), **k),
        "plan": lambda **k: sv.VerifyPlan(B, K, V, device=f"cuda:{index}", return_probs=True, **k)(
            target, draft, toks, uni),
        "sparse": lambda **k: sv.spec_verify_sparse_draft(target, t((B, K, 20), BF), cids, [1] * K, 10, toks, uni,
                                                          return_probs=True, **k),
        "shortlist": lambda **k: sv.spec_draft_head_shortlist(h, W, t((B, 2), I32), 10, **k),
        "positions": lambda **k: sv.spec_draft_head_positions(h, W, cids, [1] * K, 10, **k),
        "static": lambda **k: sv.spec_draft_head_static(h, W, ids, 10, **k),
        "kv_commit": lambda **k: sv.spec_kv_commit(t((P, B, L, 128), BF), staging, n, at, **k),
        "quantize": lambda **k: sv.spec_quantize_rows(h, **k),
        "head_quantized": lambda **k: sv.spec_draft_head_quantized(h, wc, ws, ids, 10, **k),
        "kv_commit_quantized": lambda **k: sv.spec_kv_commit_quantized(codes, scales, staging, n, at, **k),
        "kv_read_quantized": lambda **k: sv.spec_kv_read_quantized(codes, scales, at, t((P, B, L, 128), BF), **k),
        "logprobs": lambda **k: sv.spec_token_logprobs(target, t((B, K + 1), I32), 3, **k),
    }
