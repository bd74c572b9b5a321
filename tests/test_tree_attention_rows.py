"""A row of tree attention depends on its query and on what it sees, to the bit: not on the rows that
share its wave, its block or its launch, nor on when another block writes."""
import pytest
import torch

from tests.test_tree_attention import BF, DEV, F32, Case
from tests.test_tree_plans import lengths

# Rows with keys of their own to a wave and rows that share them, over one block's keys, pieces and ranges.
FORMS = {
    "own keys": dict(B=2, N=7, Hq=4, Hkv=2, D=64, L=700, lens=[700, 333]),
    "own keys, 48 rows": dict(B=1, N=12, Hq=4, Hkv=1, D=128, L=900, lens=[900]),
    "shared keys": dict(B=2, N=33, Hq=4, Hkv=1, D=64, L=800, lens=[800, 450]),
    "pieces": dict(B=1, N=7, Hq=4, Hkv=1, D=64, L=9000, lens=[9000]),
    "pieces of shared keys": dict(B=1, N=40, Hq=4, Hkv=1, D=128, L=9000, lens=[9000]),
    "ranges": dict(B=260, N=7, Hq=4, Hkv=1, D=64, L=2100, lens=lengths(260, 2100, {0: 2100, 99: 1500}, 3)),
    "ranges of shared keys": dict(B=260, N=20, Hq=4, Hkv=1, D=64, L=2100,
                                  lens=lengths(260, 2100, {0: 2100, 99: 1500}, 3)),
    "heads of 256": dict(B=1, N=7, Hq=4, Hkv=1, D=256, L=700, lens=[700]),
}


def case(form, dtype, quantized=False, parents=None):
    kw = dict(FORMS[form])
    return Case(21, dtype=dtype, quantized=quantized, parents=parents, **kw)


def tree(form):
    """Node 0 is the root of 1, 2 and 3, node 2 of 5, node 5 of 6; node 4 is absent; the others hang from 1."""
    N = FORMS[form]["N"]
    return [([-1, 0, 0, 0, -2, 2, 5] + [1] * N)[:N]] * FORMS[form]["B"]


@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("form", sorted(FORMS))
@pytest.mark.parametrize("what", ["a sibling's key", "another node's query", "an absent node", "another head's query"])
def test_a_row_depends_on_what_it_sees_alone(form, dtype, quantized, what):
    """Values that make other rows' scores large, so that their references move with many tiles."""
    c = case(form, dtype, quantized, tree(form))
    clean = c.call()
    nodes = torch.arange(c.N)
    free, heads = nodes, torch.arange(c.Hq)
    if what == "a sibling's key":
        c.k_new[:, 2] *= 30
        free = nodes[(nodes != 2) & (nodes != 5) & (nodes != 6)]
    elif what == "another node's query":
        c.q[:, 3] *= 40
        free = nodes[nodes != 3]
    elif what == "an absent node":
        c.q[:, 4] *= 40
        c.k_new[:, 4] *= 30
        c.v_new[:, 4] *= 30
    else:
        c.q[:, :, 1] *= 40
        heads = heads[heads != 1]
    got = c.call()
    assert torch.equal(got[:, free][:, :, heads], clean[:, free][:, :, heads])
    if what != "an absent node":
        assert not torch.equal(got, clean)
    assert not got[:, 4].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("form", ["own keys", "shared keys", "ranges"])
def test_special_values_of_others_change_no_bit(form, dtype):
    """As above with NaN and infinities."""
    c = case(form, dtype, False, tree(form))
    clean = c.call()
    free = [i for i in range(c.N) if i not in (2, 5, 6)]
    for t in (c.q, c.k_new, c.v_new):
        t[:, 2, :, ::3] = float("nan")
        t[:, 2, :, 1] = float("inf")
    got = c.call()
    assert torch.equal(got[:, free], clean[:, free])


@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [dict(N=20, Hq=2, Hkv=1, L=300), dict(N=12, Hq=4, Hkv=1, L=90),
                                   dict(N=33, Hq=4, Hkv=1, L=500), dict(N=50, Hq=3, Hkv=1, L=300),
                                   dict(N=63, Hq=5, Hkv=1, D=128, L=700), dict(N=9, Hq=14, Hkv=2, D=256, L=200),
                                   dict(B=260, N=11, Hq=4, Hkv=1, D=64, L=2100,
                                        lens=lengths(260, 2100, {0: 2100, 99: 1500}, 3))],
                         ids=lambda s: "-".join(str(v) for v in s.values() if isinstance(v, int)))
def test_written_over_the_queries_with_rows_left_over(shape, dtype, quantized):
    """Several blocks share a KV head's rows and the last of them has room left; one has all of the keys and
    writes its rows at once."""
    kw = dict(dict(B=3, D=64), **shape)
    kw.setdefault("lens", [kw["L"]] * kw["B"])
    c = Case(31, dtype=dtype, quantized=quantized, **kw)
    c.q *= 3
    apart = c.call()
    for _ in range(4):
        q = c.q.to(DEV)
        kept, c.q = c.q, q
        got = c.call(out=q)
        c.q = kept
        assert got is q and torch.equal(got, apart)


@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,L", [(64, 500), (128, 9000), (256, 500)])
def test_no_other_blocks_query_is_read(D, L, dtype, quantized):
    """40 rows, in groups of 32 or 16: the rows of nodes 16 to 19 are a block's that has room for more."""
    c = Case(32, B=1, N=20, Hq=2, Hkv=1, D=D, L=L, lens=[L], dtype=dtype, quantized=quantized)
    clean = c.call()
    c.q[:, 0] *= 40
    got = c.call()
    assert torch.equal(got[:, 16:], clean[:, 16:]) and not torch.equal(got[:, 0], clean[:, 0])
