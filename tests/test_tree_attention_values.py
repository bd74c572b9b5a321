"""Values and scores that are not finite: one rule wherever an entry lies, in a tile that every row sees whole or
in one at an end or at a window's edge, in the same block's keys or in another piece's."""
import numpy as np
import pytest
import torch

from tests import quant_ref as Q
from tests import tree_ref as R
from tests.test_tree_attention import BF, F32, Case
from tests.test_tree_plans import lengths

# Cached entries of the sequence under test (the last one), and how the rows get at them.
FORMS = {
    "own keys": dict(B=1, N=5, Hq=4, Hkv=1, D=64, lens=[203], L=210),
    "heads of 128": dict(B=1, N=12, Hq=4, Hkv=1, D=128, lens=[330], L=330),
    "heads of 200": dict(B=1, N=3, Hq=4, Hkv=1, D=200, lens=[203], L=210),
    "shared keys": dict(B=1, N=40, Hq=2, Hkv=1, D=64, lens=[203], L=210),
    "pieces": dict(B=1, N=5, Hq=4, Hkv=1, D=64, lens=[5003], L=5003),
    "pieces of shared keys": dict(B=1, N=40, Hq=2, Hkv=1, D=64, lens=[5003], L=5003),
    "ranges": dict(B=260, N=2, Hq=4, Hkv=1, D=16, lens=lengths(260, 2100, {259: 2100}, 1), L=2100),
}


def build(form, dtype, where):
    """Random inputs whose queries have 1 in place 0, so that a key's value there is an addend of its score."""
    c = Case(41, dtype=dtype, **FORMS[form])
    c.q[..., 0] = 1.0
    for t in (c.cache[0], c.k_new):
        t[..., 0] = 0.0
    n = int(c.lens[-1])
    at = {"first tile": 5, "mid": n // 2, "last whole tile": n // 32 * 32 - 1, "behind it": n - 1}[where]
    return c, at


def want(c, without=None):
    """The last sequence's result in 64 bits and its bound, without one of its cached entries if so asked."""
    k, v = (x[-1:] if without is None else np.delete(x[-1:], without, 1) for x in c.values())
    n = int(c.lens[-1]) - (without is not None)
    out, spread, score = R.attention(Q.as_f64(c.q)[-1:], k, v, Q.as_f64(c.k_new)[-1:], Q.as_f64(c.v_new)[-1:],
                                     c.parents.tolist()[-1:], [n], c.D ** -0.5)
    return out[0], R.attention_bound(out, spread, score, c.L + c.N, c.D, c.dtype is BF)[0]


WHERE = ["first tile", "mid", "last whole tile", "behind it"]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("where", WHERE)
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_a_value_that_is_seen(form, dtype, where, value):
    """With a weight that fp32 holds, an infinity stays one; a NaN is one."""
    c, at = build(form, dtype, where)
    c.cache[1][-1, at, 0, 3] = 0.0
    full, bound = want(c)
    c.cache[1][-1, at, 0, 3] = value
    got = Q.as_f64(c.call()[-1])
    there = (~np.isnan(got[..., 3])) & (got[..., 3] == value) if value == value else np.isnan(got[..., 3])
    seen = np.abs(full).sum(-1) > 0     # absent nodes are zeros
    assert (there | ~seen).all() and not got[~seen].any()
    others = [d for d in range(c.D) if d != 3]
    assert (np.abs(got - full)[..., others] <= bound[..., others]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("where", WHERE)
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_value_under_a_score_of_minus_infinity(form, dtype, where, value):
    """Its weight is 0, and 0 times an infinity is NaN; the entry has no other part in the row."""
    c, at = build(form, dtype, where)
    full, bound = want(c, at)
    c.cache[0][-1, at, 0, 0] = -float("inf")
    c.cache[1][-1, at, 0, 3] = value
    got = Q.as_f64(c.call()[-1])
    seen = np.abs(full).sum(-1) > 0
    assert np.isnan(got[seen][..., 3]).all() and not got[~seen].any()
    others = [d for d in range(c.D) if d != 3]
    assert (np.abs(got - full)[..., others] <= bound[..., others]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("form", sorted(FORMS))
def test_many_scores_of_minus_infinity(form, dtype):
    """More of them in a row than a wave, a block or a piece has keys, with one infinite value among them; and
    with all of them so, zeros."""
    c, _ = build(form, dtype, "mid")
    n = int(c.lens[-1])
    lo, hi = n // 8, n - n // 8
    c.cache[0][-1, lo:hi, 0, 0] = -float("inf")
    c.cache[1][-1, (lo + hi) // 2, 0, 3] = float("inf")
    got = c.call()[-1].float()
    absent = torch.tensor([line is None for line in R.lines(c.parents[-1].tolist())], device=got.device)
    assert torch.isnan(got[~absent][..., 3]).all() and not got[absent].any()
    assert torch.isfinite(got[..., [d for d in range(c.D) if d != 3]]).all()
    c.cache[0][-1, :, 0, 0] = -float("inf")
    c.k_new[-1, :, 0, 0] = -float("inf")
    assert not c.call()[-1].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("where", WHERE)
def test_an_infinity_of_a_weight_too_small_for_fp32_is_not_finite(form, dtype, where):
    c, at = build(form, dtype, where)
    c.cache[0][-1, at, 0, 0] = -1e4
    c.cache[1][-1, at, 0, 3] = float("inf")
    got = c.call()[-1]
    absent = torch.tensor([line is None for line in R.lines(c.parents[-1].tolist())], device=got.device)
    assert not torch.isfinite(got[~absent][..., 3]).any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("own", [False, True])
def test_infinities_at_a_windows_edge_and_in_the_tree(dtype, own):
    """A chain with a window: entry 33 of 40 is 7 before node 0; node 1's own entry is seen from node 1 on."""
    c = Case(43, B=1, N=6, D=64, L=40, lens=[40], parents=[[-1, 0, 1, 2, 3, 4]], dtype=dtype)
    c.q[..., 0] = 1.0
    k, v, at = (c.k_new, c.v_new, 1) if own else (*c.cache, 33)
    k[0, at, :, 0] = -float("inf")
    clean = c.call(window=9)
    v[0, at, :, 3] = float("inf")
    got = c.call(window=9)
    sees = [1, 2, 3, 4, 5] if own else [0, 1]
    blind = [i for i in range(6) if i not in sees]
    assert torch.equal(got[0, blind], clean[0, blind]) and torch.isnan(got[0, sees][..., 3]).all()
    k[0, at, :, 0] = 0.0
    got = c.call(window=9)
    assert (got[0, sees][..., 3] == float("inf")).all() and torch.isfinite(got[0, blind]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 40, 9000])
@pytest.mark.parametrize("N", [1, 40])
def test_scores_beyond_fp32_are_nan_not_a_finite_answer(dtype, N, n):
    """scale * q.k * log2(e) that overflows counts as +inf, whose softmax is NaN."""
    c = Case(44, B=1, N=N, Hq=2, Hkv=1, D=8, L=n, lens=[n], parents=[[-1] * N], dtype=dtype)
    c.q[..., 0] = 1.6e19
    c.cache[0][..., 0] = 0.0
    c.k_new[..., 0] = 0.0
    c.cache[0][0, n // 2, 0, 0] = 1.6e19
    assert torch.isnan(c.call(scale=1.0)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("N", [5, 40])
@pytest.mark.parametrize("L", [30, 4000])
def test_a_bad_length_makes_absent_nodes_nan_too(N, L):
    """A sequence whose length cannot be is NaN as a whole, as in the plain form; another's absent nodes are zeros."""
    parents = [[-1, 0, -2, 2] + [0] * (N - 4)] * 3
    c = Case(45, B=3, N=N, Hq=4, Hkv=2, L=L, lens=[L + 1, L, -1], parents=parents)
    got = c.call()
    assert torch.isnan(got[[0, 2]]).all() and torch.isfinite(got[1]).all() and not got[1, 2:4].any()
    c.check(got)
