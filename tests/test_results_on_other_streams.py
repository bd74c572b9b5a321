"""Results of a call that is given a stream other than the current one belong
to that stream: its kernels write them, and the caching allocator hands a
block out again only in its own stream's order."""
import pytest
import torch

from tests.standins import Gpus, Stream, calls

NAMES = sorted(calls())


def results(got):
    return [t for t in (got if isinstance(got, tuple) else (got,)) if t.made_on is not None]


@pytest.mark.parametrize("name", NAMES)
def test_results_are_allocated_on_the_calls_stream(monkeypatch, name):
    gpus = Gpus(monkeypatch)
    side = Stream(0)
    got = results(calls()[name](stream=side))
    assert all(t.made_on is side for t in gpus.made if t.numel()), [t.made_on for t in gpus.made]
    # the caller goes on with them on the current stream
    assert all(gpus.default[0] in t.recorded for t in got)
    assert gpus.at == gpus.default


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("explicit", [False, True])
def test_calls_on_the_current_stream(monkeypatch, name, explicit):
    gpus = Gpus(monkeypatch)
    side = Stream(0)
    with gpus.stream(side):
        got = results(calls()[name](**({"stream": side} if explicit else {})))
    assert all(t.made_on is side for t in gpus.made)
    assert not any(t.recorded for t in got)


# ---- on the GPU: the allocator's own record of whose each block is -----------------

def stream_of(t):
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no segment holds the tensor")


@pytest.mark.gpu
def test_blocks_belong_to_the_calls_stream():
    import speculative_sampling_verification_vocab_amd as sv
    dev = torch.device("cuda", 0)
    side = torch.cuda.Stream()
    x = torch.randn(6, 9, 3000, device=dev)
    t = torch.randint(0, 3000, (6, 9), device=dev, dtype=torch.int32)
    h = torch.randn(6, 256, device=dev).to(torch.bfloat16)
    ids = torch.arange(30, dtype=torch.int32, device=dev)
    n = torch.tensor([1, 2], dtype=torch.int32, device=dev)
    torch.cuda.synchronize()
    got = list(sv.spec_token_logprobs(x, t, 4, stream=side))
    codes, scales = sv.spec_quantize_rows(h, stream=side)
    got += [codes, scales, sv.spec_draft_head_quantized(h, codes, scales, ids[:6], 1, stream=side)]
    cache = torch.zeros(2, 2, 8, 128, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
    steps = torch.zeros(2, 2, 8, 1, dtype=torch.uint8, device=dev).view(torch.float8_e8m0fnu)
    staging, at = torch.zeros(2, 2, 3, 128, device=dev), torch.zeros(2, dtype=torch.int32, device=dev)
    rows = torch.zeros(2, 2, 8, 128, device=dev)
    side.wait_stream(torch.cuda.current_stream())
    got.append(sv.spec_kv_commit_quantized(cache, steps, staging, n, at, stream=side))
    got.append(sv.spec_kv_read_quantized(cache, steps, at, rows, stream=side))
    got.append(sv.spec_kv_commit(rows, staging, n, at, stream=side))
    torch.cuda.synchronize()
    assert [stream_of(v) for v in got] == [side.cuda_stream] * len(got)
    assert at.tolist() == [2, 4] and all((v == 0).all() for v in got[-3:])
