"""The Python half of the operators of a step with a tree of drafts (stand-ins,
no GPU): on which stream results are allocated, which device is current, whose
a workspace is."""
import pytest
import torch

import speculative_sampling_verification_vocab_amd as sv
from tests.standins import BF, E8, F8, F32, I32, Gpus, Stream, tensor


def calls(index=0):
    def t(shape, dtype):
        return tensor(shape, dtype, index)
    B, N, L, H, D, P = 2, 3, 8, 2, 64, 4
    q, new = t((B, N, 4, D), BF), t((B, N, H, D), BF)
    par, n = t((B, N), I32), t((B,), I32)
    kv, codes, scales = t((B, L, H, D), BF), t((B, L, H, D), F8), t((B, L, 1), E8)
    tok = t((B, N), I32)
    staging = t((P, B, N, H, D), BF)
    return {
        "attention": lambda **k: sv.spec_tree_attention(q, kv, kv, new, new, par, n, **k),
        "attention_quantized": lambda **k: sv.spec_tree_attention_quantized(q, codes, scales, codes, scales, new, new,
                                                                            par, n, **k),
        "sample": lambda **k: sv.spec_sample_tokens(t((B, N, 50), BF), t((B, N), F32), **k),
        "commit": lambda **k: sv.spec_tree_commit(t((P, B, L, H, D), BF), staging, tok, par, tok, n, **k),
        "commit_quantized": lambda **k: sv.spec_tree_commit_quantized(
            t((P, B, L, H, D), F8), t((P, B, L, 1), E8), staging, tok, par, tok, n, **k),
    }


NAMES = sorted(calls())


@pytest.mark.parametrize("name", NAMES)
def test_results_are_allocated_on_the_calls_stream(monkeypatch, name):
    gpus = Gpus(monkeypatch)
    side = Stream(0)
    got = calls()[name](stream=side)
    got = got if isinstance(got, tuple) else (got,)
    assert all(t.made_on is side for t in gpus.made if t.numel())
    assert all(gpus.default[0] in t.recorded for t in got)
    with gpus.stream(side):
        before = len(gpus.made)
        calls()[name]()
        assert all(t.made_on is side and not t.recorded for t in gpus.made[before:])


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("own,current", [(0, 0), (1, 0), (0, 1), (1, 1)])
def test_the_tensors_device_is_current(monkeypatch, name, own, current):
    gpus = Gpus(monkeypatch)
    gpus.dev = current
    side = Stream(own)
    calls(own)[name]()
    calls(own)[name](stream=side)
    assert [dev for _, dev, _ in gpus.lib.calls] == [own] * 2
    assert [side.cuda_stream in args for _, _, args in gpus.lib.calls] == [False, True]
    assert all(t.device.index == own for t in gpus.made) and gpus.dev == current


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(monkeypatch, name):
    gpus = Gpus(monkeypatch)
    with pytest.raises(ValueError):
        calls(0)[name](stream=Stream(1))
    assert not gpus.lib.calls


@pytest.mark.parametrize("name", ["attention", "attention_quantized"])
def test_captured_calls_own_their_workspace(monkeypatch, name):
    gpus = Gpus(monkeypatch)
    monkeypatch.setattr(sv, "_default_ws", {})

    def scratch():
        return [t for t in gpus.made if t.dtype == torch.uint8 and t.numel() >= gpus.need]
    side = Stream(0)
    with gpus.stream(side):
        gpus.captured.append(side)
        calls()[name]()
        calls()[name]()
        gpus.captured.clear()
        assert len(scratch()) == 2 and sv._default_ws == {}
        calls()[name]()
        calls()[name]()
        assert len(scratch()) == 3
