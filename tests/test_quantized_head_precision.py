"""How exactly the quantised head adds its products, in each of its tiles.

Products of two e4m3 codes have at most 8 significant bits, times a power of two.

fp32 outputs: products are exact and added in fp32.  A sum of d products is off
by at most d roundings of half a step, 2^-24 of a partial sum; for products of
random signs a partial sum is no larger than the result (rms over all outputs),
and roundings add in quadrature: the rms error is at most sqrt(d) * 2^-24 of
the results' rms.  That is 5.4e-6 at d = 8192, 6.7e-7 at d = 128; the 8-bit matrix
instruction, whose rms error is 1.4e-5 of it, would fail.

bf16 outputs: of each 8 consecutive dims the 8-bit matrix instruction drops what
lies below 2^-13 of the largest product's power of two, toward zero.  The
largest itself keeps all 8 bits, so a group of 8 is off by at most 7 * 2^-13 of
its largest product; d / 8 + 16 additions of groups, wave groups and slices by
one step, 2^-23 of the sum of magnitudes; then half a step of bf16, 2^-8."""
import numpy as np
import pytest
import torch

from tests.test_quantized_head import BF, DEV, F32, sv

pytestmark = pytest.mark.gpu

# each tile and its own-h form, with and without a split of d, one to 64 blocks of 128
SHAPES = [(5, 4096, 8016), (12, 4096, 600), (12, 2048, 9000), (24, 1024, 700), (32, 384, 17000), (50, 8192, 300),
          (64, 640, 34000), (100, 128, 500), (128, 4096, 3000), (100, 384, 66000), (300, 640, 26000)]


def values(codes, scales):
    """float64 on the GPU: what the codes stand for."""
    step = scales.double().repeat_interleave(128, -1)
    return codes.double() * step


def normal(M, d, V, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    h = torch.randn(M, d, generator=g, device=DEV).to(BF)
    W = (torch.randn(V, d, generator=g, device=DEV) * d ** -0.5).to(BF)
    codes, scales = sv().spec_quantize_rows(W)
    hv, wv = values(*sv().spec_quantize_rows(h)), values(codes, scales)
    ids = torch.arange(V, dtype=torch.int32, device=DEV)
    return h, codes, scales, ids, hv, wv.t().contiguous()


@pytest.mark.parametrize("M,d,V", SHAPES)
def test_fp32_outputs_are_sums_in_fp32(M, d, V):
    print(f"case M={M} d={d} V={V}", flush=True)
    h, codes, scales, ids, hv, wt = normal(M, d, V, M + d)
    want = hv @ wt
    err = sv().spec_draft_head_quantized(h, codes, scales, ids, 1, dtype=F32).double() - want
    rms = want.pow(2).mean().sqrt().item()
    assert err.pow(2).mean().sqrt().item() <= d ** 0.5 * 2.0 ** -24 * rms
    assert torch.all(err.abs() <= (d + 16) * 2.0 ** -23 * (hv.abs() @ wt.abs()))


@pytest.mark.parametrize("M,d,V", SHAPES)
def test_bf16_outputs(M, d, V):
    print(f"case M={M} d={d} V={V}", flush=True)
    h, codes, scales, ids, hv, wt = normal(M, d, V, M + d + 1)
    want = hv @ wt
    err = sv().spec_draft_head_quantized(h, codes, scales, ids, 1, dtype=BF).double() - want
    rms = want.pow(2).mean().sqrt().item()
    # the cuts in quadrature: sqrt(7 d / 8) * 2^-13 of a group's largest product, some four times sqrt(1 / d) of the
    # result; below 2^-11 of it
    assert err.pow(2).mean().sqrt().item() <= (2.0 ** -8 + 2.0 ** -11) * rms
    mag = hv.abs() @ wt.abs()
    assert torch.all(err.abs() <= (7 * 2.0 ** -13 + (d / 8 + 16) * 2.0 ** -23) * mag + 2.0 ** -8 * want.abs())


def outliers(M, d, V):
    """Rows whose groups of 8 dims each hold one large value, which cancels with that of the next group: what is left
    is the sum of the small ones."""
    g = torch.Generator(device=DEV).manual_seed(77)
    h = torch.randn(M, d, generator=g, device=DEV)
    W = torch.randn(V, d, generator=g, device=DEV)
    at = 3 + 8 * torch.arange(d // 8, device=DEV)
    sign = 1.0 - 2.0 * (torch.arange(d // 8, device=DEV) % 2)
    h[:, at] = 64.0 * sign
    W[:, at] = 32.0
    h, W = h.to(BF), W.to(BF)
    codes, scales = sv().spec_quantize_rows(W)
    hv, wv = values(*sv().spec_quantize_rows(h)), values(codes, scales)
    assert torch.equal(hv[:, at], (64.0 * sign).double().expand(M, -1)) and (wv[:, at] == 32.0).all()
    ids = torch.arange(V, dtype=torch.int32, device=DEV)
    return h, codes, scales, ids, hv, wv


@pytest.mark.parametrize("M,d,V", [(5, 512, 64), (16, 1024, 200), (24, 1024, 64), (60, 512, 140), (130, 512, 200)])
def test_outliers_that_cancel(M, d, V):
    h, codes, scales, ids, hv, wv = outliers(M, d, V)
    p = hv[:, None, :] * wv[None, :, :]
    want, mag = p.sum(-1), p.abs().sum(-1)
    most = p.abs().unflatten(-1, (-1, 8)).amax(-1).sum(-1)
    f32 = sv().spec_draft_head_quantized(h, codes, scales, ids, 1, dtype=F32).double()
    assert torch.all((f32 - want).abs() <= (d + 16) * 2.0 ** -23 * mag)
    bf16 = sv().spec_draft_head_quantized(h, codes, scales, ids, 1, dtype=BF).double()
    tol = 7 * 2.0 ** -13 * most + (d / 8 + 16) * 2.0 ** -23 * mag + 2.0 ** -8 * want.abs()
    assert torch.all((bf16 - want).abs() <= tol)


def test_a_second_segment_of_scales():
    """More than 32 blocks of 128 in the 128 x 256 tile: scales are put in LDS twice, the starts staggered in each."""
    M, d, V = 100, 4224, 66000
    h, codes, scales, ids, hv, wt = normal(M, d, V, 5)
    # blocks of one row at very different scales: one taken from a neighbour shows
    g = torch.Generator(device=DEV).manual_seed(6)
    shift = torch.randint(-4, 5, (V, d // 128), generator=g, device=DEV)
    scales = (scales.view(torch.uint8).int() + shift).to(torch.uint8).view(torch.float8_e8m0fnu)
    wt = values(codes, scales).t().contiguous()
    want, mag = hv @ wt, hv.abs() @ wt.abs()
    for out in (F32, BF):
        err = (sv().spec_draft_head_quantized(h, codes, scales, ids, 1, dtype=out).double() - want).abs()
        tol = (d + 16) * 2.0 ** -23 * mag if out == F32 else \
            (7 * 2.0 ** -13 + (d / 8 + 16) * 2.0 ** -23) * mag + 2.0 ** -8 * want.abs()
        assert torch.all(err <= tol)
        assert err.pow(2).mean().sqrt() <= (d ** 0.5 * 2.0 ** -24 if out == F32 else 2.0 ** -8 + 2.0 ** -11) * \
            want.pow(2).mean().sqrt()


@pytest.mark.parametrize("M,d,V", [(128, 4096, 33000), (300, 640, 26000), (5, 4096, 8016)])
def test_same_on_every_call_in_large_grids(M, d, V):
    """Bit for bit, with other products on the chip in between."""
    h, codes, scales, ids, _, _ = normal(M, d, V, 9)
    other = torch.flip(ids, (0,)).contiguous()
    for out in (BF, F32):
        first = sv().spec_draft_head_quantized(h, codes, scales, ids, 1, dtype=out)
        for _ in range(4):
            sv().spec_draft_head_quantized(h.flip(0).contiguous(), codes, scales, other, 1, dtype=out)
            assert torch.equal(sv().spec_draft_head_quantized(h, codes, scales, ids, 1, dtype=out), first)


def test_tiles_are_the_ones_meant():
    """The shapes above reach every tile of the plan (its rule, from its sizes)."""
    def tile(M, N):
        def tiles(a, b):
            return -(-M // a) * -(-N // b)
        if M <= 64:
            return 0 if M <= 16 else 1 if M <= 32 else 2
        if M <= 128:
            return 4 if tiles(128, 256) >= 256 else 3
        return 5 if tiles(256, 256) >= 200 else 3
    assert {tile(M, V) for M, _, V in SHAPES} == set(range(6))
    assert tile(100, 66000) == 4 and np.ceil(4224 / 128) > 32
