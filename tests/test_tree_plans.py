"""How a call's work is cut: keys shared out over blocks in pieces and ranges,
rows that share their keys, several planes with one walk.  The sizes are those
where each way of cutting begins; bounds are those of the operators' own tests."""
import pytest
import torch

from tests.test_tree_attention import BF, DEV, F32, Case, poison, shifted, sv
from tests.test_tree_commit import Case as Commit


def lengths(B, L, some, seed=0):
    """Mostly short sequences, and `some` at their places."""
    g = torch.Generator().manual_seed(seed)
    n = torch.randint(0, 40, (B,), generator=g)
    for b, v in some.items():
        n[b] = v
    return n


def space(*shape):
    return sv()._native.load().spec_tree_attention_workspace_bytes(*shape, 1)


# ---- ranges ---------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("some", [{}, {0: 2100}, {259: 2100}, {3: 2100, 4: 2099, 64: 2100, 128: 1000, 258: 64}])
def test_batches_with_few_long_sequences(dtype, some, quantized):
    """More sequences than lanes, on blocks that have parts of many of them or of one."""
    B, L = 260, 2100
    c = Case(len(some), B=B, N=2, Hq=2, Hkv=1, D=8, L=L, lens=lengths(B, L, some), dtype=dtype, quantized=quantized)
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,Hq", [(1, 2), (5, 6), (9, 8), (17, 8), (64, 8)])
def test_ranges_over_heads_and_rows(dtype, N, Hq, quantized):
    """Two KV heads, 1 to 256 rows each, every sequence cut somewhere else."""
    B, L = 130, 2300
    some = {0: 2300, 1: 0, 2: 517, 77: 2050, 129: 1601}
    c = Case(N, B=B, N=N, Hq=Hq, Hkv=2, D=16, L=L, lens=lengths(B, L, some, N), dtype=dtype, quantized=quantized)
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("quantized", [False, True])
def test_ranges_of_whole_heads(D, quantized):
    B, L = 260, 2080
    c = Case(D, B=B, N=20, Hq=4, Hkv=1, D=D, L=L, lens=lengths(B, L, {17: 2080, 200: 900}), quantized=quantized)
    c.check()


@pytest.mark.gpu
def test_ranges_with_bad_lengths():
    B, L = 260, 2100
    n = lengths(B, L, {5: -1, 64: 2 ** 31 - 1, 65: L + 1, 66: L, 259: -2 ** 31})
    c = Case(1, B=B, N=3, Hq=1, Hkv=1, D=8, L=L, lens=n, dtype=F32)
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 3), (700, 70), (1500, 700), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_ranges_with_windows(window, sinks):
    """A window leaves few keys, so pieces; a wide one with sinks ranges in three parts."""
    B, L = 260, 2400
    n = lengths(B, L, {0: 2400, 100: 2222, 101: 1800, 259: 1200})
    Case(2, B=B, N=4, Hq=2, Hkv=1, D=8, L=L, lens=n, dtype=F32).check(window=window, sinks=sinks)


@pytest.mark.gpu
def test_a_sequence_alone_gives_what_the_batch_gives():
    """Within the bounds of both; and the same call gives the same bits."""
    B, L = 260, 2100
    c = Case(6, B=B, N=2, Hq=2, Hkv=1, D=64, L=L, lens=lengths(B, L, {7: 2100}))
    got = c.call()
    assert torch.equal(got, c.call())
    one = Case(6, B=B, N=2, Hq=2, Hkv=1, D=64, L=L, lens=lengths(B, L, {7: 2100}))
    for name in ("q", "k_new", "v_new", "parents", "lens"):
        setattr(one, name, getattr(one, name)[7:8])
    one.cache = [t[7:8] for t in one.cache]
    one.B = 1
    one.check()
    one.check(got[7:8])


# ---- pieces ---------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("L", [1020, 1022, 1023, 1024, 1279, 1500])
def test_where_pieces_begin(dtype, L):
    """Two nodes: pieces from 1025 keys on."""
    assert (space(3, 2, 4, 2, 64, L) > 0) == (L + 2 > 1024)
    Case(L, B=3, N=2, Hq=4, Hkv=2, D=64, L=L, lens=[L, 0, L // 2], dtype=dtype).check()


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 40])
def test_more_pieces_than_tiles(N):
    """An almost empty cache with room for many keys."""
    c = Case(N, B=2, N=N, Hq=4, Hkv=2, D=128, L=9000, lens=[3, 0])
    assert space(2, N, 4, 2, 128, 9000) > 0
    c.check()


# ---- shared keys ----------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("D", [64, 72, 128])
@pytest.mark.parametrize("n", [0, 1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300])
def test_lengths_around_the_shared_stages(n, D, quantized):
    Case(n + D, B=2, N=33, Hq=6, Hkv=3, D=D, L=max(n, 1) + 5, lens=[n, max(0, n - 2)], quantized=quantized).check()


@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("window", [1, 63, 64, 65, 150])
@pytest.mark.parametrize("sinks", [0, 1, 63, 64, 100])
def test_windows_around_the_shared_stages(window, sinks, quantized):
    c = Case(window + sinks, B=2, N=35, Hq=2, Hkv=1, D=128, L=310, lens=[310, 190], quantized=quantized)
    c.check(window=window, sinks=sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [0, 17, 64, 100, 130])
def test_unused_entries_of_shared_keys_may_hold_anything(n):
    c = Case(n, B=1, N=40, Hq=2, Hkv=1, D=128, L=140, lens=[n])
    clean = c.call(), c.call(window=45, sinks=2)
    for t in c.cache:
        poison(t, (0, slice(n, None)))
    assert torch.equal(c.call(), clean[0])
    for t in c.cache:
        poison(t, (0, slice(2, max(2, n - 44))))
    assert torch.equal(c.call(window=45, sinks=2), clean[1])


@pytest.mark.gpu
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_bad_value_in_a_whole_stage_reaches_every_row(value):
    c = Case(3, B=1, N=40, Hq=2, Hkv=1, D=64, L=200, lens=[200])
    c.cache[1][0, 70, 0, 5] = value
    c.check()


@pytest.mark.gpu
def test_values_that_begin_between_whole_pieces():
    """A cache off by one value can not go to shared memory in 16-byte pieces."""
    c = Case(5, B=2, N=40, Hq=2, Hkv=1, D=128, L=1500, lens=[1500, 777])
    t = [x.to(DEV) for x in (c.q, c.k_new, c.v_new, c.parents, c.lens)]
    for by in [(1, 0), (0, 1), (1, 1)]:
        k, v = (shifted(x.to(DEV), b) for x, b in zip(c.cache, by))
        c.check(sv().spec_tree_attention(t[0], k, v, *t[1:]))


# ---- in place -------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("B,N,L,lens", [(2, 5, 90, None), (2, 40, 300, None), (1, 40, 5000, [4990]), (260, 3, 2100, None)])
def test_the_output_may_be_the_queries(B, N, L, lens):
    lens = lengths(B, L, {B - 1: L}) if lens is None else lens
    c = Case(B, B=B, N=N, Hq=2, Hkv=1, D=64, L=L, lens=lens)
    want = c.call()
    t = [x.to(DEV) for x in (c.q, *c.cache, c.k_new, c.v_new, c.parents, c.lens)]
    got = sv().spec_tree_attention(*t, out=t[0])
    assert got is t[0] and torch.equal(got, want)


# ---- planes ---------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("P,B,E", [(17, 1024, 8), (67, 1024, 8), (41, 2048, 3), (130, 128, 128)])
def test_several_planes_with_one_walk(P, B, E, in_place, quantized):
    """Two to eight planes a block, the last block with fewer."""
    Commit(P, P=P, B=B, N=5, L=7, E=E, quantized=quantized, kinds=2).check(in_place)
