"""Rows, weights and batches of more than 2^32 values: the last ones against the
same values on their own, and the longest row that is accepted."""
import math

import pytest
import torch

from tests.test_quantized_rows_and_cache import sv

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
BF, F32 = torch.bfloat16, torch.float32


def noise(shape, dtype, seed, step=1 << 26):
    """Normal values, made piece by piece."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.empty(shape, dtype=dtype, device=DEV)
    flat = x.view(-1)
    for i in range(0, flat.numel(), step):
        flat[i:i + step] = torch.randn(min(step, flat.numel() - i), generator=g, device=DEV).to(dtype)
    return x


def test_rows():
    x = noise((140001, 32768), BF, 1)
    codes, scales = sv().spec_quantize_rows(x)
    for at in (0, 65536, 131072, 140001 - 7):      # values 0, 2^31, 2^32 and the last
        c, s = sv().spec_quantize_rows(x[at:at + 7].contiguous())
        assert torch.equal(codes.view(torch.uint8)[at:at + 7], c.view(torch.uint8))
        assert torch.equal(scales.view(torch.uint8)[at:at + 7], s.view(torch.uint8))


@pytest.mark.parametrize("M", [5, 40, 100, 300])
def test_head_on_a_large_weight(M):
    """Codes of 4.5 GB; the shortlist takes rows from both of its ends."""
    V, d, cs = 1100000, 4096, 100
    g = torch.Generator(device=DEV).manual_seed(2)
    codes = torch.randint(0, 126, (V, d), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.randint(112, 118, (V, d // 128), generator=g, device=DEV, dtype=torch.uint8)
    ids = torch.tensor([0, 5242, 5243, 10485, 10486, 10999], dtype=torch.int32, device=DEV)
    rows = (ids.long()[:, None] * cs + torch.arange(cs, device=DEV)).flatten()
    h = noise((M, d), BF, 3)
    f8, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    own = torch.arange(6, dtype=torch.int32, device=DEV)
    for out in (BF, F32):
        got = sv().spec_draft_head_quantized(h, codes.view(f8), scales.view(e8), ids, cs, dtype=out)
        want = sv().spec_draft_head_quantized(h, codes[rows].view(f8), scales[rows].view(e8), own, cs, dtype=out)
        assert torch.equal(got, want)


def test_head_with_many_outputs():
    """2.6e9 logits."""
    M, d, V = 20001, 128, 128256
    h = noise((M, d), BF, 4)
    W = sv().spec_quantize_rows(noise((V, d), BF, 5))
    ids = torch.arange(V, dtype=torch.int32, device=DEV)
    got = sv().spec_draft_head_quantized(h, *W, ids, 1, dtype=BF)
    for at in (0, 16742, 20001 - 300):             # from outputs 0, 2^31 and the last ones
        want = sv().spec_draft_head_quantized(h[at:at + 300].contiguous(), *W, ids, 1, dtype=BF)
        assert torch.equal(got[at:at + 300], want)


@pytest.mark.parametrize("N,V,dtype", [(17001, 262144, BF), (140001, 32768, F32)])
def test_log_probabilities(N, V, dtype):
    """The two launches of long rows and the one of short ones."""
    x = noise((N, V), dtype, 6)
    t = torch.arange(N, dtype=torch.int32, device=DEV) % V
    got = sv().spec_token_logprobs(x, t, 5)
    n = 1000 if dtype == BF else 300               # enough for the same launch geometry: sums are grouped alike
    for at in (0, (1 << 31) // V, N - n):
        one = sv().spec_token_logprobs(x[at:at + n].contiguous(), t[at:at + n].contiguous(), 5)
        assert torch.equal(one[2], got[2][at:at + n])
        for a, b in ((one[i], got[i][at:at + n]) for i in (0, 1, 3)):
            assert torch.all((a - b).abs() <= 2.0 ** -24 * (64 + 4 * b.abs()))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_longest_row(dtype):
    V = 1 << 30
    x = noise((1, V), dtype, 7)
    best = torch.tensor([V - 1, 3, V // 2 + 1, V // 2, V - 4096], device=DEV)
    x[0, best] = torch.tensor([30.0, 29.0, 28.0, 27.0, 26.0], device=DEV).to(dtype)
    z = s = 0.0                                    # sums of e^(x - 30) and of that times x, in 64 bits
    for i in range(0, V, 1 << 26):
        p = x[0, i:i + (1 << 26)].double()
        e = torch.exp(p - 30.0)
        z, s = z + e.sum().item(), s + (e * p).sum().item()
    lse = 30.0 + math.log(z)
    entropy = lse - s / z
    for tok in (V - 1, 12345):
        lp, ent, ids, tops = sv().spec_token_logprobs(x, torch.tensor([tok], dtype=torch.int32, device=DEV), 5)
        assert ids[0].tolist() == best.tolist()
        for got, want in [(lp[0].item(), x[0, tok].item() - lse), (ent[0].item(), entropy)] + \
                list(zip(tops[0].tolist(), [v - lse for v in (30.0, 29.0, 28.0, 27.0, 26.0)])):
            assert abs(got - want) <= 2.0 ** -24 * (64 + 4 * abs(want)), (got, want)
