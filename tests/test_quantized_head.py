"""Drafter head on a weight in the 8-bit block format against a 64-bit product
of the values that the codes stand for.

Tolerance: products of two e4m3 values with power-of-two scales are exact in
fp32; a sum of d of them in fp32, in any order, is off by at most d roundings,
each of at most one step (2^-23, which also covers truncation) of a partial
sum that the sum of magnitudes bounds: (d + 16) * 2^-23 * sum |h w|, 16 for
the sums of wave groups and slices.  bf16 output adds 2^-8 of the value."""
import ctypes

import numpy as np
import pytest
import torch

from tests import quant_ref as R

DEV = torch.device("cuda", 0)
BF, F32 = torch.bfloat16, torch.float32


def sv():
    import speculative_sampling_verification_vocab_amd as m
    return m


def case(M, d, V, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    h = (torch.randn(M, d, generator=g) * torch.exp(spread * torch.randn(M, 1, generator=g))).to(BF)
    W = (torch.randn(V, d, generator=g) * torch.exp(spread * torch.randn(V, 1, generator=g)) * d ** -0.5).to(BF)
    # blocks of one row at very different scales: a scale taken from a neighbour shows
    W *= torch.exp2(torch.randint(-4, 5, (V, -(-d // 128)), generator=g).float()).repeat_interleave(128, 1)[:, :d]
    return h, W.to(BF)


def product(h, W, rows):
    """float64 (values, sums of magnitudes) on the GPU (fp64 product)."""
    hv = torch.from_numpy(R.values(*R.quantize(R.as_f64(h)))).to(DEV)
    wv = torch.from_numpy(R.values(*R.quantize(R.as_f64(W)))).to(DEV)
    live = rows >= 0
    wv = wv[torch.from_numpy(np.where(live, rows, 0)).to(DEV)]
    wv[torch.from_numpy(~live).to(DEV)] = 0.0
    wt = wv.t().contiguous()
    return (hv @ wt).cpu().numpy(), (hv.abs() @ wt.abs()).cpu().numpy()


def check(M, d, V, cs, ids, out, seed=1):
    h, W = case(M, d, V, seed)
    ids = np.asarray(ids, dtype=np.int32)
    rows = (ids.astype(np.int64)[:, None] * cs + np.arange(cs)).reshape(-1)
    rows[np.repeat((ids < 0) | (ids >= V // cs), cs)] = -1
    want, mag = product(h, W, rows)
    codes, scales = sv().spec_quantize_rows(W.to(DEV))
    got = sv().spec_draft_head_quantized(h.to(DEV), codes, scales, torch.from_numpy(ids).to(DEV), cs, dtype=out)
    torch.cuda.synchronize()
    assert got.shape == (M, len(ids) * cs) and got.dtype == out
    err = np.abs(R.as_f64(got) - want)
    tol = (d + 16) * 2.0 ** -23 * mag + (2.0 ** -8 * np.abs(want) if out == BF else 0.0)
    worst = np.max(err - tol) if err.size else 0.0
    assert worst <= 0.0, (worst, np.argwhere(err > tol)[:5])
    assert np.all(R.as_f64(got)[:, rows < 0] == 0.0)
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,d,V,cs,n", [
    (1, 1, 1, 1, 1), (1, 128, 40, 1, 33), (5, 256, 999, 9, 100), (16, 1000, 512, 1, 512), (17, 384, 700, 7, 30),
    (32, 130, 96, 3, 32), (33, 2048, 300, 1, 131), (64, 640, 1000, 1, 65), (65, 1152, 260, 2, 129),
    (128, 4096, 400, 1, 400), (130, 512, 5000, 10, 385), (257, 200, 130, 1, 127), (2, 8192, 128, 1, 100),
    (3, 8576, 64, 1, 64), (70, 16512, 200, 1, 130)])
def test_products(M, d, V, cs, n, out):
    """Rows, columns and dims that end inside a tile, one to many blocks of 128, each tile and the split over d."""
    print(f"case M={M} d={d} V={V} cs={cs} n={n} {out}", flush=True)
    g = torch.Generator().manual_seed(V)
    check(M, d, V, cs, torch.randperm(V // cs, generator=g)[:n].numpy(), out)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [4, 100])
def test_ids_out_of_range_and_repeated(M):
    got = check(M, 384, 600, 4, [3, -1, 149, 150, 3, 0, 2147483647, -2147483648, 7], F32)
    assert torch.equal(got[:, 0:4], got[:, 16:20])


@pytest.mark.gpu
@pytest.mark.parametrize("M,d,V", [(5, 4096, 24000), (40, 2048, 17000), (200, 1024, 36000), (100, 384, 66000),
                                   (300, 640, 26000), (513, 1024, 17410), (129, 4224, 52000),
                                   (2, 8448, 8300), (16, 4096, 9000), (9, 3200, 8200), (5, 4095, 8200), (1, 23000, 8200)])
def test_wide_shortlists(M, d, V):
    """Grids of many tiles, without a split."""
    check(M, d, V, 1, np.arange(V - 3), BF)


@pytest.mark.gpu
def test_scales_at_their_ends():
    """Rows whose blocks sit at the ends of the scale's range, and zeros."""
    h = torch.zeros(4, 512, dtype=BF)
    W = torch.zeros(40, 512, dtype=BF)
    h[0, :128], W[:, :128] = 2.0 ** 60, 2.0 ** 60
    h[1, 128:256], W[:, 128:256] = 2.0 ** -60, 2.0 ** -60
    h[2, 300] = 1.0
    W[:, 300] = torch.arange(40).to(BF)
    want, mag = product(h, W, np.arange(40))
    codes, scales = sv().spec_quantize_rows(W.to(DEV))
    got = sv().spec_draft_head_quantized(h.to(DEV), codes, scales, torch.arange(40, dtype=torch.int32, device=DEV), 1)
    err = np.abs(R.as_f64(got) - want)
    assert np.all(err <= (512 + 16) * 2.0 ** -23 * mag)


@pytest.mark.gpu
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M", [3, 40])
def test_small_weights(M, out):
    """Weights down to 2^-118, whose smallest codes stand for values below the normal range of bf16 and fp32."""
    h, W = case(M, 512, 90, 12)
    W = (W.float() * 2.0 ** -112).to(BF)
    want, mag = product(h, W, np.arange(90))
    codes, scales = sv().spec_quantize_rows(W.to(DEV))
    got = sv().spec_draft_head_quantized(h.to(DEV), codes, scales, torch.arange(90, dtype=torch.int32, device=DEV), 1,
                                         dtype=out)
    err = np.abs(R.as_f64(got) - want)
    # flushing what lies below the normal range would cost 2^-126 |h| a product
    tol = (512 + 16) * 2.0 ** -23 * mag + (2.0 ** -8 * np.abs(want) if out == BF else 0.0) + 2.0 ** -133
    flushed = 2.0 ** -126 * np.abs(R.as_f64(h)).sum(1, keepdims=True)
    assert np.all(err <= tol + flushed)


@pytest.mark.gpu
def test_nan_stays_in_its_row():
    h, W = case(6, 256, 50, 9)
    h[2, 17] = float("nan")
    W[31, 200] = float("inf")
    codes, scales = sv().spec_quantize_rows(W.to(DEV))
    got = sv().spec_draft_head_quantized(h.to(DEV), codes, scales, torch.arange(50, dtype=torch.int32, device=DEV), 1)
    bad = torch.isnan(got).cpu().numpy()
    want = np.zeros((6, 50), dtype=bool)
    want[2, :] = want[:, 31] = True
    assert np.array_equal(bad, want)


@pytest.mark.gpu
def test_same_on_every_call_and_leading_dims():
    h, W = case(12, 1024, 700, 4)
    codes, scales = sv().spec_quantize_rows(W.to(DEV))
    ids = torch.arange(700, dtype=torch.int32, device=DEV)
    a = sv().spec_draft_head_quantized(h.view(3, 4, 1024).to(DEV), codes, scales, ids, 1)
    b = sv().spec_draft_head_quantized(h.to(DEV), codes, scales, ids, 1, out=torch.empty(12, 700, device=DEV))
    assert a.shape == (3, 4, 700) and torch.equal(a.view(12, 700), b)
    assert sv().spec_draft_head_quantized(h[:0].to(DEV), codes, scales, ids, 1).shape == (0, 700)
    assert sv().spec_draft_head_quantized(h.to(DEV), codes, scales, ids[:0], 1).shape == (12, 0)


@pytest.mark.gpu
def test_unaligned_outputs_and_scales():
    """Outputs and scale rows that begin off 16 and 4 bytes."""
    h, W = case(20, 512, 64, 6)
    codes, scales = sv().spec_quantize_rows(W.to(DEV))
    ids = torch.arange(64, dtype=torch.int32, device=DEV)
    want = sv().spec_draft_head_quantized(h.to(DEV), codes, scales, ids, 1)
    sbuf = torch.empty(scales.numel() + 1, dtype=torch.uint8, device=DEV)
    sbuf[1:] = scales.view(torch.uint8).flatten()
    obuf = torch.full((20 * 64 + 2,), 5.0, device=DEV)
    out = obuf[1:-1].view(20, 64)
    sv().spec_draft_head_quantized(h.to(DEV), codes, sbuf[1:].view(64, 4).view(torch.float8_e8m0fnu), ids, 1, out=out)
    assert torch.equal(out, want) and obuf[0] == 5.0 and obuf[-1] == 5.0


# ---- refusals -----------------------------------------------------------------------

OK, INVALID, UNSUP, WS = 0, 1, 2, 3


def test_refusals():
    from speculative_sampling_verification_vocab_amd import _native
    lib, p = _native.load(), ctypes.c_void_p
    size = lib.spec_draft_head_quantized_workspace_bytes
    ok = dict(h=0x10000, wc=0x20000, ws_=0x30001, ids=0x40000, M=4, d=256, V=1000, cs=10, n=20, out=0x50000, dt=0,
              work=0x100000, wb=1 << 30)

    def call(**o):
        a = {**ok, **o}
        return lib.spec_draft_head_quantized(p(a["h"]), p(a["wc"]), p(a["ws_"]), p(a["ids"]), a["M"], a["d"], a["V"],
                                             a["cs"], a["n"], p(a["out"]), a["dt"], p(a["work"]), a["wb"], None)
    for name in ("h", "wc", "ws_", "ids", "out"):
        assert call(**{name: None}) == INVALID, name
    assert call(M=-1) == INVALID and call(d=0) == INVALID and call(V=0) == INVALID and call(cs=0) == INVALID
    assert call(n=-1) == INVALID and call(n=101) == INVALID and call(dt=4) == INVALID
    assert call(cs=7) == UNSUP
    assert call(h=0x10001) == INVALID and call(wc=0x20008) == INVALID and call(ids=0x40002) == INVALID
    assert call(out=0x50002) == INVALID and call(out=0x50001, dt=1) == INVALID
    need = size(40, 256, 1000, 10, 20)
    assert need >= 40 * 256 + 40 * 2
    for o in (dict(work=None), dict(work=0x100080), dict(wb=need - 1)):
        assert call(M=40, **o) == WS
    assert size(4, 256, 1000, 10, 20) == 0                # few values of h: none needed
    assert call(M=0, h=None) == OK and call(n=0, out=None) == OK
    assert call(M=0x7fffffff, d=128, V=1 << 20, cs=1, n=1 << 20) == UNSUP
    assert call(d=0x7fffffff) == UNSUP
    assert size(0, 256, 1000, 10, 20) == 0 and size(4, 256, 1000, 7, 20) == 0 and size(4, 0, 1000, 10, 20) == 0


def test_cpu_tensors_are_refused():
    W = torch.zeros(4, 128, dtype=torch.uint8).view(torch.float8_e4m3fn)
    s = torch.zeros(4, 1, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    with pytest.raises(ValueError):
        sv().spec_draft_head_quantized(torch.zeros(2, 128, dtype=BF), W, s, torch.zeros(1, dtype=torch.int32), 1)


@pytest.mark.gpu
def test_shapes_and_types_are_checked():
    h, W = case(4, 256, 60, 2)
    h = h.to(DEV)
    codes, scales = sv().spec_quantize_rows(W.to(DEV))
    ids = torch.arange(6, dtype=torch.int32, device=DEV)
    f = sv().spec_draft_head_quantized
    for a in ((h.float(), codes, scales, ids, 1), (h[:, :100].contiguous(), codes, scales, ids, 1),
              (h, codes.view(torch.uint8), scales, ids, 1), (h, codes, scales[:59], ids, 1),
              (h, codes, scales, ids.long(), 1), (h, codes, scales, ids.view(2, 3), 1), (h.t(), codes, scales, ids, 1),
              (h, codes, scales, ids.cpu(), 1)):
        with pytest.raises(ValueError):
            f(*a)
    with pytest.raises(ValueError):
        f(h, codes, scales, ids, 1, dtype=torch.float16)
    with pytest.raises(ValueError):
        f(h, codes, scales, ids, 1, out=torch.empty(4, 7, device=DEV))
    for cs in (0, -1, 7):
        with pytest.raises((sv().SpecVerifyError, ValueError, RuntimeError)):
            f(h, codes, scales, ids, cs)
