"""A row of tree attention depends on its query and on what it sees, to the bit: not on the queries of
another block, nor on when that block writes."""
import pytest
import torch

from tests.test_tree_attention import BF, DEV, F32, Case
from tests.test_tree_plans import lengths


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
