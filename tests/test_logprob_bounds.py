"""Log-probabilities are at most 0 and entropies at least 0, also where one
token has (nearly) all of the probability and the roundings of the sums could
carry a result past its bound."""
import numpy as np
import pytest
import torch

from tests.test_token_logprobs import BF, DEV, F32, INF, compare, sv

pytestmark = pytest.mark.gpu


def bounded(x, t, T=1.0):
    got = [v.cpu().numpy() for v in sv().spec_token_logprobs(x.to(DEV), t.to(DEV), 3, T)]
    live = ~np.isnan(got[0])
    assert live.any()
    assert (got[0][live] <= 0).all(), got[0][live].max()
    assert (got[1][live] >= 0).all(), got[1][live].min()
    assert (got[3][live] <= 0).all(), got[3][live].max()
    return got


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,V", [(300, 5000), (40, 70001), (900, 33000)])
def test_one_token_left(N, V, dtype):
    """A mask that leaves one token: probability 1, entropy 0, for that token and seen from another."""
    g = torch.Generator().manual_seed(V)
    x = torch.full((N, V), -INF)
    at = torch.arange(N) * 7 % V
    x[torch.arange(N), at] = torch.randn(N, generator=g) * 20
    x = x.to(dtype)
    for T in (1.0, 0.37):
        T = float(np.float32(T))
        for t in (at, (at + 1) % V):
            t = t.to(torch.int32)
            got = bounded(x, t, T)
            compare(x[:6], t[:6], 3, T, [v[:6] for v in got])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,V", [(400, 5000), (40, 70001)])
def test_one_token_far_above_the_rest(N, V, dtype):
    """The rest is too small to be seen in 32 bits; the row's token is the likeliest one or up to 13 below it."""
    g = torch.Generator().manual_seed(V + 1)
    x = torch.randn(N, V, generator=g)
    at = torch.arange(N) * 7 % V
    low = (at + 5) % V
    x[torch.arange(N), at] = 80 + torch.rand(N, generator=g)
    x[torch.arange(N), low] = 80 - 13 * torch.rand(N, generator=g)
    x = x.to(dtype)
    for t in (at, low):
        t = t.to(torch.int32)
        got = bounded(x, t)
        compare(x[:6], t[:6], 3, 1.0, [v[:6] for v in got])
    x[torch.arange(N), low] = 0.0
    bounded(x, at.to(torch.int32))
