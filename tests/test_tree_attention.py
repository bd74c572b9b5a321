"""Attention of a draft tree over the cache, of values and 8-bit, against a plain
one in 64 bits; bounds are those of tree_ref.attention_bound."""
import ctypes

import numpy as np
import pytest
import torch

from tests import quant_ref as Q
from tests import tree_ref as R

DEV = torch.device("cuda", 0)
BF, F32 = torch.bfloat16, torch.float32
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def sv():
    import speculative_sampling_verification_vocab_amd as m
    return m


class Case:
    """Random inputs (on the CPU in their types) and what they give in 64 bits."""

    def __init__(self, seed, B=2, N=5, Hq=4, Hkv=2, D=64, L=50, dtype=BF, quantized=False, lens=None, parents=None):
        g = torch.Generator().manual_seed(seed)
        self.B, self.N, self.Hq, self.Hkv, self.D, self.L, self.dtype, self.quantized = \
            B, N, Hq, Hkv, D, L, dtype, quantized

        def rand(*shape):
            return torch.randn(shape, generator=g).to(dtype)
        self.q, self.k_new, self.v_new = rand(B, N, Hq, D), rand(B, N, Hkv, D), rand(B, N, Hkv, D)
        if quantized:
            nb = -(-Hkv * D // 128)
            self.codes = [torch.randint(0, 256, (B, L, Hkv, D), generator=g, dtype=torch.uint8) for _ in range(2)]
            for c in self.codes:
                c[(c & 127) == 127] = 3
            self.scales = [torch.randint(116, 120, (B, L, nb), generator=g, dtype=torch.uint8) for _ in range(2)]
        else:
            self.cache = [rand(B, L, Hkv, D) for _ in range(2)]
        if parents is None:
            parents = torch.tensor([[int(torch.randint(-1, i, (1,), generator=g)) if i else -1 for i in range(N)]
                                    for _ in range(B)]).view(B, N)
        self.parents = torch.as_tensor(parents, dtype=torch.int32)
        if lens is None:
            lens = torch.randint(0, L + 1, (B,), generator=g)
        self.lens = torch.as_tensor(lens, dtype=torch.int32)

    def values(self):
        """The cache's keys and values as float64 arrays."""
        if not self.quantized:
            return [Q.as_f64(c) for c in self.cache]
        shape = (self.B, self.L, self.Hkv, self.D)
        return [Q.values(c.flatten(2).numpy(), s.numpy()).reshape(shape) for c, s in zip(self.codes, self.scales)]

    def call(self, **kw):
        t = [x.to(DEV) for x in (self.q, self.k_new, self.v_new, self.parents, self.lens)]
        if self.quantized:
            (kc, vc), (ks, vs) = ([c.to(DEV).view(F8) for c in self.codes], [s.to(DEV).view(E8) for s in self.scales])
            return sv().spec_tree_attention_quantized(t[0], kc, ks, vc, vs, *t[1:], **kw)
        return sv().spec_tree_attention(t[0], self.cache[0].to(DEV), self.cache[1].to(DEV), *t[1:], **kw)

    def check(self, got=None, scale=None, window=0, sinks=0):
        scale = self.D ** -0.5 if scale is None else scale
        if got is None:
            got = self.call(scale=scale, window=window, sinks=sinks)
        k, v = self.values()
        want, spread, score = R.attention(Q.as_f64(self.q), k, v, Q.as_f64(self.k_new), Q.as_f64(self.v_new),
                                          self.parents.tolist(), self.lens.tolist(), scale, window, sinks)
        got = Q.as_f64(got)
        assert got.shape == want.shape
        special = ~np.isfinite(want)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(got[special & ~np.isnan(want)], want[special & ~np.isnan(want)])
        bound = R.attention_bound(want, spread, score, self.L + self.N, self.D, self.dtype is BF)
        off = np.abs(np.where(special, 0.0, got) - np.where(special, 0.0, want))
        ok = special | (off <= bound)
        assert ok.all(), (np.argwhere(~ok)[:5], off[~ok][:5], bound[~ok][:5])
        return want


# ---- shapes ---------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [8, 40, 64, 72, 96, 128, 136, 192, 256])
@pytest.mark.parametrize("N,L", [(1, 33), (7, 70), (64, 5)])
def test_head_sizes(dtype, D, N, L, quantized):
    Case(D + N, N=N, D=D, L=L, Hq=6, Hkv=3, dtype=dtype, quantized=quantized).check()


@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 1), (16, 1), (17, 1), (40, 8), (7, 7), (64, 2)])
@pytest.mark.parametrize("N", [1, 3, 16, 64])
def test_head_counts_and_rows(dtype, Hq, Hkv, N, quantized):
    Case(Hq * N, B=1, N=N, Hq=Hq, Hkv=Hkv, D=64, L=45, dtype=dtype, quantized=quantized).check()


@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 511, 512, 513, 2047, 2600])
def test_lengths(dtype, n, quantized):
    """Lengths around tiles, blocks and splits, in a cache with room behind and in one that is full."""
    Case(n, B=2, N=3, L=max(n, 1) + 37, lens=[n, max(0, n - 1)], dtype=dtype, quantized=quantized).check()
    Case(n, B=1, N=2, Hkv=1, D=128, L=n, lens=[n], dtype=dtype, quantized=quantized).check()


@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_cache_in_splits(dtype, quantized):
    c = Case(3, B=1, N=4, Hq=4, Hkv=1, D=128, L=20011, lens=[20000], dtype=dtype, quantized=quantized)
    assert sv()._native.load().spec_tree_attention_workspace_bytes(1, 4, 4, 1, 128, 20011, 1) > 0
    c.check()


@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [1e-30, 0.5, 3.0])
def test_scales_and_peaked_rows(dtype, scale, quantized):
    """From all keys alike to rows that one key decides, with the largest score anywhere."""
    c = Case(11, N=6, D=64, L=300, lens=[300, 299], dtype=dtype, quantized=quantized)
    c.check(scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rising", [False, True])
def test_references_that_move_with_every_tile(dtype, rising):
    c = Case(12, B=1, N=2, Hq=2, Hkv=1, D=64, L=1500, lens=[1500], dtype=dtype)
    c.q[:] = 1.0
    ramp = torch.linspace(-30, 30, 1500)
    c.cache[0][0, :, 0] = ((ramp if rising else -ramp)[:, None] * torch.ones(64) / 8).to(dtype)
    c.check(scale=0.125)


# ---- trees ----------------------------------------------------------------------

CHAIN = [[i - 1 for i in range(64)]]
TREES = {
    "chain of 64": CHAIN,
    "all roots": [[-1] * 40],
    "star": [[-1] + [0] * 50],
    "binary": [[-1] + [(i - 1) // 2 for i in range(1, 63)]],
    "absent nodes": [[-1, -2, 0, 1, 2, 3, 5, 0, 64, -7, 9, 2147483647, -2147483648, 13, 0]],
    "all absent": [[-2] * 9],
    "only the last": [[-2] * 8 + [-1]],
    "self and later parents": [[0, -1, 3, 1, 4, 1, 9, 6, 8]],
}


@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("name", sorted(TREES))
@pytest.mark.parametrize("n", [0, 77])
def test_trees(name, n, quantized):
    parents = TREES[name]
    c = Case(5, B=1, N=len(parents[0]), L=77, lens=[n], parents=parents, dtype=F32, quantized=quantized)
    want = c.check()
    absent = [line is None for line in R.lines(parents[0])]
    assert not want[0, absent].any()
    c.check(window=9, sinks=2)


@pytest.mark.gpu
def test_a_chain_is_causal_attention():
    """Node i of a chain sees the cache and the nodes up to itself: torch's own attention with such a mask."""
    c = Case(6, B=2, N=9, D=64, L=40, lens=[40, 40], parents=[list(range(-1, 8))] * 2, dtype=F32)
    got = c.call()
    k, v = (torch.cat([x.double(), y.double()], 1).repeat_interleave(2, 2) for x, y in zip(c.cache, (c.k_new, c.v_new)))
    mask = torch.arange(49)[None, :] <= 40 + torch.arange(9)[:, None]
    x = torch.einsum("bihd,bjhd->bhij", c.q.double(), k) / 8.0
    p = torch.softmax(x.masked_fill(~mask, -float("inf")), -1)
    want = torch.einsum("bhij,bjhd->bihd", p, v)
    assert (got.cpu().double() - want).abs().max() < 3e-6


# ---- windows --------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [1, 2, 31, 32, 64, 150, 2 ** 31 - 1])
@pytest.mark.parametrize("sinks", [0, 1, 40, 2 ** 31 - 1])
def test_windows(dtype, window, sinks, quantized):
    Case(window % 97 + sinks % 89, B=4, N=20, L=203, lens=[0, 1, 60, 203], dtype=dtype,
         quantized=quantized).check(window=window, sinks=sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(700, 0), (700, 33), (5, 900)])
def test_windows_in_long_caches(window, sinks):
    Case(8, B=2, N=12, L=3001, lens=[3001, 1500], dtype=F32).check(window=window, sinks=sinks)


# ---- what is not seen -----------------------------------------------------------

def poison(t, where):
    """NaN, infinities and the type's ends at `where` of t."""
    bad = torch.tensor([float("nan"), float("inf"), -float("inf"), torch.finfo(t.dtype).max, torch.finfo(t.dtype).min])
    t[where] = bad[torch.arange(t[where].numel()) % 5].to(t.dtype).view(t[where].shape)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [0, 17, 64, 100])
@pytest.mark.parametrize("D", [64, 128, 200, 256])
def test_unused_entries_may_hold_anything(dtype, n, D):
    """The cache behind a sequence's length, entries that the window hides from every node, and absent nodes."""
    c = Case(n, B=1, N=6, D=D, L=130, lens=[n], parents=[[-1, 0, -2, 2, 1, 1]], dtype=dtype)
    clean = c.call(), c.call(window=9, sinks=2)
    for t in c.cache:
        poison(t, (0, slice(n, None)))
    for t in (c.q, c.k_new, c.v_new):
        poison(t, (0, slice(2, 4)))
    assert torch.equal(c.call(), clean[0])
    for t in c.cache:
        poison(t, (0, slice(2, max(2, n - 9))))
    assert torch.equal(c.call(window=9, sinks=2), clean[1])
    c.check(c.call(window=9, sinks=2), window=9, sinks=2)


@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
def test_unused_codes_may_be_nan(quantized):
    c = Case(4, B=1, N=3, D=128, L=70, lens=[37], quantized=True)
    clean = c.call()
    for t in c.codes:
        t[0, 37:] = 127
    for t in c.scales:
        t[0, 37:] = 255 if quantized else 0
    assert torch.equal(c.call(), clean)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("what", ["k", "v", "both"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_a_bad_node_reaches_its_descendants_alone(dtype, what, value):
    """Node 2 is bad; 4 and 5 descend from it; 0, 1, 3 and 6 do not see it."""
    parents = [[-1, 0, 0, 1, 2, 4, 3]]
    c = Case(9, B=1, N=7, D=64, L=40, lens=[40], parents=parents, dtype=dtype)
    clean = c.call()
    for t in [c.k_new] * (what != "v") + [c.v_new] * (what != "k"):
        t[0, 2, 0, ::7] = value
    got = c.call()
    free = [0, 1, 3, 6]
    assert torch.equal(got[0, free], clean[0, free])
    assert torch.equal(got[0, :, 2:], clean[0, :, 2:])     # the other KV head's queries
    c.check(got)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_bad_cache_entry_reaches_the_nodes_whose_window_has_it(dtype, value):
    """A chain with a window: entry 33 is at a distance of 7 from node 0, 8 from node 1, ..."""
    c = Case(10, B=1, N=6, D=64, L=40, lens=[40], parents=[[-1, 0, 1, 2, 3, 4]], dtype=dtype)
    clean = c.call(window=9)
    c.cache[1][0, 33, :, 3] = value
    got = c.call(window=9)
    assert torch.equal(got[0, 2:], clean[0, 2:])
    assert not torch.isfinite(got[0, :2, :, 3]).any()
    c.check(got, window=9)


@pytest.mark.gpu
def test_bad_codes_in_a_window():
    c = Case(13, B=1, N=4, D=128, L=40, lens=[40], parents=[[-1, 0, 1, 2]], quantized=True)
    clean = c.call(window=9)
    c.codes[1][0, 33, :, 5] = 127   # seen by nodes 0 and 1
    got = c.call(window=9)
    assert torch.equal(got[0, 2:], clean[0, 2:]) and torch.isnan(got[0, :2, :, 5]).all()
    c.codes[1][0, 33, :, 5] = 0
    c.scales[0][0, 32] = 255        # keys seen by node 0 alone
    got = c.call(window=9)
    assert torch.isnan(got[0, 0]).all() and torch.isfinite(got[0, 1:]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_scores_of_minus_infinity(dtype):
    """Rows whose every score is -inf are zeros; one other score decides a row."""
    c = Case(14, B=1, N=2, Hq=2, Hkv=1, D=64, L=5, lens=[5], parents=[[-1, -1]], dtype=dtype)
    c.q[:] = 1.0
    c.cache[0][:] = 0.0
    c.cache[0][0, :, 0, 0] = -float("inf")
    c.k_new[:] = 0.0
    c.k_new[0, :, 0, 0] = torch.tensor([-float("inf"), 2.0])
    got = c.call()
    assert not got[0, 0].any()
    assert torch.equal(got[0, 1], c.v_new[0, 1].to(DEV).expand(2, 64))


@pytest.mark.gpu
@pytest.mark.parametrize("split", [False, True])
def test_bad_lengths_give_nan_for_their_sequence(split):
    L = 4000 if split else 30
    c = Case(15, B=4, N=3, L=L, lens=[L + 1, 30, -1, -2 ** 31], dtype=F32)
    got = c.call(window=2 ** 31 - 1)
    assert torch.isnan(got[[0, 2, 3]]).all()
    c.lens[[0, 2, 3]] = 0
    assert torch.equal(got[1], c.call(window=2 ** 31 - 1)[1])


# ---- buffers --------------------------------------------------------------------

def shifted(t, by):
    """t's values in memory that begins `by` elements into a buffer."""
    b = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    b[by:] = t.flatten()
    return b[by:].view(t.shape)


@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [72, 128])
def test_any_alignment_of_whole_elements(dtype, D, quantized):
    c = Case(16, N=5, D=D, L=90, dtype=dtype, quantized=quantized)
    want = c.call()
    q, kn, vn, par, n = (shifted(t.to(DEV), 1) for t in (c.q, c.k_new, c.v_new, c.parents, c.lens))
    out = shifted(torch.zeros_like(c.q).to(DEV), 3)
    if quantized:
        kc, vc = (shifted(t.to(DEV), 1).view(F8) for t in c.codes)
        ks, vs = (shifted(t.to(DEV), 1).view(E8) for t in c.scales)
        got = sv().spec_tree_attention_quantized(q, kc, ks, vc, vs, kn, vn, par, n, out=out)
    else:
        got = sv().spec_tree_attention(q, *(shifted(t.to(DEV), 1) for t in c.cache), kn, vn, par, n, out=out)
    assert got is out and torch.equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("L", [30, 5000])
def test_only_the_output_is_written(L):
    """Guards around the output and the workspace stay as they were, and inputs too."""
    c = Case(17, B=2, N=3, L=L, dtype=BF)
    guard = torch.full((c.q.numel() + 512,), 7.0, dtype=BF, device=DEV)
    out = guard[256:256 + c.q.numel()].view(c.q.shape)
    lib = sv()._native.load()
    need = lib.spec_tree_attention_workspace_bytes(2, 3, c.Hq, c.Hkv, c.D, L, 1)
    assert (need > 0) == (L == 5000)
    ws = sv().Workspace(DEV)
    ws.buf = torch.full((need + 4096,), 77, dtype=torch.uint8, device=DEV)
    ws._stream = torch.cuda.current_stream()
    kept = [t.clone() for t in (c.q, *c.cache, c.k_new, c.v_new)]
    c.check(c.call(out=out, workspace=ws))
    assert (guard[:256] == 7).all() and (guard[256 + c.q.numel():] == 7).all()
    assert (ws.buf[need:] == 77).all()
    assert all(torch.equal(a, b) for a, b in zip(kept, (c.q, *c.cache, c.k_new, c.v_new)))


@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
def test_the_same_on_every_call(quantized):
    c = Case(18, B=3, N=17, Hq=8, Hkv=2, D=128, L=6000, quantized=quantized)
    first = c.call()
    for _ in range(4):
        assert torch.equal(c.call(), first)


@pytest.mark.gpu
def test_empty_calls():
    for kw in (dict(B=0), dict(N=0)):
        c = Case(19, **kw)
        assert c.call().shape == c.q.shape


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    """The last sequence's keys and values begin more than 2^32 bytes into their planes (8-bit, 6.6 GB each)."""
    B, L, Hkv, D = 3, 16800, 512, 256
    assert 2 * L * Hkv * D > 2 ** 32
    codes = torch.zeros((2, B, L, Hkv, D), dtype=torch.uint8, device=DEV)
    codes[:, 2, 5:9, 511] = torch.randint(0, 120, (2, 4, D), generator=torch.Generator().manual_seed(1),
                                          dtype=torch.uint8).to(DEV)
    scales = torch.full((2, B, L, Hkv * D // 128), 127, dtype=torch.uint8, device=DEV)
    q = torch.ones((B, 1, Hkv, D), dtype=BF, device=DEV)
    new = torch.zeros((B, 1, Hkv, D), dtype=BF, device=DEV)
    n = torch.tensor([0, 0, 9], dtype=torch.int32, device=DEV)
    par = torch.full((B, 1), -1, dtype=torch.int32, device=DEV)
    got = sv().spec_tree_attention_quantized(q, codes[0].view(F8), scales[0].view(E8), codes[1].view(F8),
                                             scales[1].view(E8), new, new, par, n, scale=1e-3)
    k, v = (Q.values(codes[i, 2, :9, 511].cpu().numpy(), np.full((9, 2), 127)) for i in (0, 1))
    x = np.append(k.sum(1) * 1e-3, 0.0)
    p = np.exp(x - x.max())
    want = (p[:9, None] * v).sum(0) / p.sum()
    spread = (p[:9, None] * np.abs(v)).sum(0) / p.sum()
    off = np.abs(Q.as_f64(got[2, 0, 511]) - want)
    assert (off <= R.attention_bound(want, spread, np.abs(k).sum(1).max() * 1e-3, 10, D, True)).all()
    assert not got[:2].any() and not got[2, 0, :511].any()


# ---- refusals (CPU) ---------------------------------------------------------------

FAKE = 0x10000


def c_call(quantized=False, **over):
    a = dict(q=FAKE, k=FAKE, ks=FAKE, v=FAKE, vs=FAKE, kn=FAKE, vn=FAKE, par=FAKE, n=FAKE, B=2, N=3, Hq=4, Hkv=2, D=64,
             L=5000, scale=0.125, window=0, sinks=0, dt=1, out=FAKE, ws=None, wsb=0)
    a.update(over)
    lib = sv()._native.load()
    p = {k: ctypes.c_void_p(v) if isinstance(v, int) and k in ("q k ks v vs kn vn par n out ws".split()) else v
         for k, v in a.items()}
    head = [p["q"], p["k"], p["ks"], p["v"], p["vs"]] if quantized else [p["q"], p["k"], p["v"]]
    fn = lib.spec_tree_attention_quantized if quantized else lib.spec_tree_attention
    return fn(*head, p["kn"], p["vn"], p["par"], p["n"], a["B"], a["N"], a["Hq"], a["Hkv"], a["D"], a["L"],
              ctypes.c_float(a["scale"]), a["window"], a["sinks"], a["dt"], p["out"], p["ws"], a["wsb"], None)


@pytest.mark.parametrize("quantized", [False, True])
def test_host_validation(quantized):
    INVALID, UNSUP, WS = 1, 2, 3

    def call(**o):
        return c_call(quantized, **o)
    assert call() == WS                                        # valid, but for the workspace
    for name in ("q", "k", "v", "kn", "vn", "par", "n", "out") + (("ks", "vs") if quantized else ()):
        assert call(**{name: None}) == INVALID, name
    for name in ("q", "kn", "vn", "out") + (() if quantized else ("k", "v")):
        assert call(**{name: FAKE + 1}) == INVALID, name       # not on an element's boundary
    assert call(par=FAKE + 2) == INVALID and call(n=FAKE + 1) == INVALID
    for o in (dict(B=-1), dict(N=-1), dict(Hq=0), dict(Hkv=0), dict(D=0), dict(L=-1), dict(dt=2), dict(window=-1),
              dict(sinks=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(**o) == INVALID, o
    for o in (dict(N=65), dict(D=60), dict(D=264), dict(Hq=5), dict(L=(1 << 30) + 1),
              dict(Hkv=1 << 17, Hq=1 << 17, D=64), dict(B=0x7fffffff), dict(Hq=1 << 23, Hkv=1)):
        assert call(**o) == UNSUP, o
    need = sv()._native.load().spec_tree_attention_workspace_bytes(2, 3, 4, 2, 64, 5000, 1)
    assert need > 0
    assert call(ws=FAKE, wsb=need - 1) == WS and call(ws=FAKE + 128, wsb=need) == WS
    assert call(B=0, q=None) == 0 and call(N=0, q=None) == 0   # nothing to do
    size = sv()._native.load().spec_tree_attention_workspace_bytes
    assert size(2, 3, 4, 2, 64, 30, 1) == 0 and size(2, 65, 4, 2, 64, 5000, 1) == 0 and size(0, 3, 4, 2, 64, 5000, 1) == 0


def test_python_refusals(monkeypatch):
    from tests.standins import Gpus, tensor
    gpus = Gpus(monkeypatch)

    def call(quantized=False, **over):
        t = dict(q=((2, 3, 4, 64), BF), k=((2, 9, 2, 64), F8 if quantized else BF),
                 v=((2, 9, 2, 64), F8 if quantized else BF), kn=((2, 3, 2, 64), BF), vn=((2, 3, 2, 64), BF),
                 par=((2, 3), torch.int32), n=((2,), torch.int32), ks=((2, 9, 1), E8), vs=((2, 9, 1), E8))
        kw = {k: over.pop(k) for k in list(over) if k in ("window", "sinks", "out", "scale")}
        t.update(over)
        x = {k: tensor(*v) for k, v in t.items()}
        tail = (x["kn"], x["vn"], x["par"], x["n"])
        if quantized:
            return sv().spec_tree_attention_quantized(x["q"], x["k"], x["ks"], x["v"], x["vs"], *tail, **kw)
        return sv().spec_tree_attention(x["q"], x["k"], x["v"], *tail, **kw)
    assert call().shape == (2, 3, 4, 64) and call(True).shape == (2, 3, 4, 64)
    made = len(gpus.lib.calls)
    for over in (dict(q=((2, 3, 4, 64), torch.float16)), dict(q=((2, 3, 256), BF)), dict(k=((2, 9, 2, 64), F32)),
                 dict(v=((2, 8, 2, 64), BF)), dict(k=((2, 9, 2, 32), BF)), dict(k=((3, 9, 2, 64), BF)),
                 dict(kn=((2, 4, 2, 64), BF)), dict(vn=((2, 3, 2, 64), F32)), dict(par=((2, 3), torch.int64)),
                 dict(par=((3, 2), torch.int32)), dict(n=((3,), torch.int32)), dict(n=((2, 1), torch.int32)),
                 dict(window=-1), dict(sinks=-1), dict(window=1 << 31), dict(sinks=1 << 31),
                 dict(out=tensor((2, 3, 4, 64), F32)), dict(out=tensor((2, 3, 256), BF))):
        with pytest.raises(ValueError):
            call(**over)
    for over in (dict(ks=((2, 9, 2), E8)), dict(vs=((2, 9, 1), torch.uint8)), dict(k=((2, 9, 2, 64), BF))):
        with pytest.raises(ValueError):
            call(True, **over)
    assert len(gpus.lib.calls) == made
    with pytest.raises(ValueError):   # no CPU path
        sv().spec_tree_attention(*[torch.zeros(1)] * 7)
