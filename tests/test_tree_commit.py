"""The walk along a tree and the commit of its path, to a cache of values and to
the 8-bit one, against a loop."""
import ctypes

import numpy as np
import pytest
import torch

from tests import quant_ref as Q
from tests import tree_ref as R

DEV = torch.device("cuda", 0)
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def sv():
    import speculative_sampling_verification_vocab_amd as m
    return m


class Case:
    def __init__(self, seed, P=2, B=5, N=9, L=30, E=64, dtype=BF, quantized=False, kinds=3, shift=0):
        g = torch.Generator().manual_seed(seed)
        self.P, self.B, self.N, self.L, self.E, self.dtype, self.quantized = P, B, N, L, E, dtype, quantized

        def place(t):
            """t on the GPU, `shift` elements into its memory."""
            b = torch.empty(t.numel() + shift, dtype=t.dtype, device=DEV)
            b[shift:] = t.flatten().to(DEV)
            return b[shift:].view(t.shape)
        self.staging = place(torch.randn((P, B, N, E), generator=g).to(dtype))
        self.nb = -(-E // 128)
        if quantized:
            self.codes = place(torch.randint(0, 256, (P, B, L, E), generator=g, dtype=torch.uint8))
            self.scales = place(torch.randint(0, 256, (P, B, L, self.nb), generator=g, dtype=torch.uint8))
        else:
            self.cache = place(torch.randn((P, B, L, E), generator=g).to(dtype))
        parents = torch.tensor([[-1 if i == 0 else int(torch.randint(0, i, (1,), generator=g)) for i in range(N)]
                                for _ in range(B)], dtype=I32).view(B, N)
        self.parents = parents
        self.tokens = torch.randint(0, kinds, (B, N), generator=g).to(I32)
        self.sampled = torch.randint(0, kinds, (B, N), generator=g).to(I32)
        self.len = torch.randint(0, max(L - N, 0) + 1, (B,), generator=g).to(I32)

    def call(self, in_place=False, planes=None):
        """Outputs as lists, the new lengths, and the cache before the call."""
        P = slice(None) if planes is None else slice(planes)
        tok, par, sam, n = (t.to(DEV) for t in (self.tokens, self.parents, self.sampled, self.len))
        new = None if in_place else torch.full_like(n, -77)
        if self.quantized:
            self.before = self.codes.clone(), self.scales.clone()
            got = sv().spec_tree_commit_quantized(self.codes[P].view(F8), self.scales[P].view(E8), self.staging[P], tok,
                                                  par, sam, n, new_len=new)
        else:
            self.before = (self.cache.clone(),)
            got = sv().spec_tree_commit(self.cache[P], self.staging[P], tok, par, sam, n, new_len=new)
        if not in_place:
            assert torch.equal(n.cpu(), self.len)
        return [t.tolist() for t in got], (n if in_place else new).tolist()

    def check(self, in_place=False):
        (acc, out, path, status), new = self.call(in_place)
        N = self.N
        want = [t.cpu().clone() for t in self.before]
        staging = Q.as_f64(self.staging)
        paths = []
        for b in range(self.B):
            p, e = R.walk(self.tokens[b].tolist(), self.parents[b].tolist(), self.sampled[b].tolist())
            paths.append(p)
            n = int(self.len[b])
            st = 2 if not p else 0 if 0 <= n <= self.L - len(p) else 1
            assert acc[b] == len(p) - 1 and path[b] == p + [-1] * (N - len(p)) and out[b] == e + [-1] * (N - len(e))
            assert status[b] == st and new[b] == (n + len(p) if st == 0 else n)
            if st == 0 and self.quantized:
                c, s = Q.quantize(staging[:, b, p])
                want[0][:, b, n:n + len(p)] = torch.from_numpy(c[..., :self.E])
                want[1][:, b, n:n + len(p)] = torch.from_numpy(s)
            elif st == 0:
                want[0][:, b, n:n + len(p)] = self.staging.cpu()[:, b, p]
        if self.quantized:
            assert Q.same_codes(self.codes.cpu().numpy(), want[0].numpy())
            assert torch.equal(self.scales.cpu(), want[1])
        else:
            assert torch.equal(self.cache.cpu(), want[0])
        return paths


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("E", [1, 2, 7, 8, 64, 100, 128, 136, 576, 1024])
def test_entry_sizes(dtype, E, quantized, in_place):
    Case(E, E=E, dtype=dtype, quantized=quantized).check(in_place)


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("N", [1, 2, 3, 33, 63, 64])
@pytest.mark.parametrize("kinds", [1, 2, 1000])
def test_tree_sizes(N, kinds, quantized, in_place):
    Case(N * kinds, N=N, B=17, L=70, kinds=kinds, quantized=quantized).check(in_place)


@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("E", [128, 1000])
def test_chains_that_are_accepted_whole(dtype, E, quantized):
    """Paths of 64 nodes, longer than a grid's blocks take at once."""
    c = Case(1, B=2, P=3, N=64, L=64, E=E, dtype=dtype, quantized=quantized)
    c.parents[:] = torch.arange(-1, 63, dtype=I32)
    c.sampled[:, :-1] = c.tokens[:, 1:]
    c.len[:] = 0
    assert [len(p) for p in c.check()] == [64, 64]


@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
def test_any_alignment_of_whole_elements(quantized):
    for dtype in (BF, F32):
        for E in (64, 100):
            Case(2, E=E, dtype=dtype, quantized=quantized, shift=3).check()


@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_faults_and_room(quantized, in_place):
    """Sequences of every kind beside each other: padded, a bad root, a bad draw on the path and off it, full, too full,
    lengths out of range."""
    c = Case(3, B=11, N=6, L=8, quantized=quantized, kinds=1)
    c.parents[:] = torch.arange(-1, 5, dtype=I32)      # a chain that is accepted whole: 6 entries
    c.len[:] = torch.tensor([0, 0, 0, 0, 0, 2, 3, -1, 2 ** 31 - 1, -2 ** 31, 9], dtype=I32)
    c.parents[0] = -2
    c.parents[1, 0] = 0
    c.sampled[2, 3] = -1
    c.sampled[3, 2], c.sampled[3, 4] = 5, -1           # the walk ends before the bad draw
    c.sampled[4, 0] = -1
    (acc, _, _, status), new = c.call(in_place)
    assert status == [2, 2, 2, 0, 2, 0, 1, 1, 1, 1, 1]
    assert acc == [-1, -1, -1, 2, -1, 5, 5, 5, 5, 5, 5]
    c = Case(3, B=11, N=6, L=8, quantized=quantized, kinds=1)
    c.parents[:] = torch.arange(-1, 5, dtype=I32)
    c.len[:] = torch.tensor([0, 0, 0, 0, 0, 2, 3, -1, 2 ** 31 - 1, -2 ** 31, 9], dtype=I32)
    c.parents[0] = -2
    c.parents[1, 0] = 0
    c.sampled[2, 3] = -1
    c.sampled[3, 2], c.sampled[3, 4] = 5, -1
    c.sampled[4, 0] = -1
    c.check(in_place)


@pytest.mark.gpu
def test_siblings_with_one_token_and_parents_out_of_range():
    """Of equal siblings the first is taken, and the second's subtree is not; nodes with a bad parent are nobody's child."""
    c = Case(4, B=1, N=9)
    c.parents[0] = torch.tensor([-1, 0, 0, 2, 1, -2, 64, 2147483647, 7], dtype=I32)
    c.tokens[0] = torch.tensor([9, 5, 5, 6, 8, 5, 5, 5, 5], dtype=I32)
    c.sampled[0] = torch.tensor([5, 6, 6, 6, 6, 6, 6, 6, 6], dtype=I32)
    assert c.check() == [[0, 1]]
    c.tokens[0, 4] = 6
    assert c.check() == [[0, 1, 4]]
    c.parents[0, 1] = 1      # its own parent
    assert c.check() == [[0, 2, 3]]


@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_without_planes_or_room(quantized, in_place):
    """P = 0 (the walk alone), a cache of no rows, entries of no values."""
    for kw in (dict(P=0), dict(L=0), dict(E=0)):
        Case(5, quantized=quantized, **kw).check(in_place)


@pytest.mark.gpu
def test_the_same_walk_as_without_planes():
    c = Case(6, B=40, N=20, kinds=2)
    a = c.call()
    b = c.call(planes=0)
    assert a == b


@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
def test_values_that_are_not_finite(quantized):
    c = Case(7, E=256, quantized=quantized)
    c.staging[:, :, :, 3] = float("nan")
    c.staging[:, :, :, 130] = float("inf")
    (_, _, path, status), new = c.call()
    for b in range(c.B):
        n = len([i for i in path[b] if i >= 0])
        at = int(c.len[b])
        rows = c.staging[:, b, path[b][:n]]
        if quantized:
            got = c.codes[:, b, at:at + n].cpu().numpy()
            assert Q.same_codes(got, Q.quantize(Q.as_f64(rows))[0])
        else:
            assert torch.equal(c.cache[:, b, at:at + n].view(torch.int16), rows.view(torch.int16))


@pytest.mark.gpu
def test_chains_agree_with_the_verify_steps_commit():
    """A chain whose root and first n drafts are accepted: spec_kv_commit of n + 1 entries."""
    c = Case(8, P=3, B=6, N=5, E=72, kinds=2)
    c.parents[:] = torch.arange(-1, 4, dtype=I32)
    other = c.cache.clone()
    (acc, _, _, _), new = c.call()
    n = c.len.to(DEV).clone()
    sv().spec_kv_commit(other, c.staging, torch.tensor(acc, dtype=I32, device=DEV) + 1, n)
    assert torch.equal(other, c.cache) and n.tolist() == new


@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
def test_offsets_beyond_32_bits(quantized):
    """The last plane begins more than 2^32 bytes into the cache."""
    P, B, N, L, E = 3, 2, 4, 4096, (1 << 18) if quantized else (1 << 17)
    cache = torch.zeros((P, B, L, E), dtype=torch.uint8 if quantized else BF, device=DEV)
    assert cache[0].numel() * cache.element_size() * 2 >= 2 ** 32
    staging = torch.randn((P, B, N, E), generator=torch.Generator(DEV).manual_seed(1), device=DEV).to(BF)
    par = torch.tensor([[-1, 0, 0, 2]] * B, dtype=I32, device=DEV)
    tok = torch.tensor([[0, 1, 2, 3]] * B, dtype=I32, device=DEV)
    sam = torch.tensor([[2, 9, 3, 9]] * B, dtype=I32, device=DEV)   # 0, 2, 3
    n = torch.tensor([L - 3, L - 3], dtype=I32, device=DEV)
    new = torch.empty_like(n)
    rows = staging[2, 1, [0, 2, 3]]
    if quantized:
        scales = torch.zeros((P, B, L, E // 128), dtype=torch.uint8, device=DEV)
        sv().spec_tree_commit_quantized(cache.view(F8), scales.view(E8), staging, tok, par, sam, n, new_len=new)
        c, s = sv().spec_quantize_rows(rows)
        assert torch.equal(cache[2, 1, L - 3:], c.view(torch.uint8)) and torch.equal(scales[2, 1, L - 3:], s.view(torch.uint8))
    else:
        sv().spec_tree_commit(cache, staging, tok, par, sam, n, new_len=new)
        assert torch.equal(cache[2, 1, L - 3:], rows)
    assert new.tolist() == [L, L] and not cache[:, :, :L - 3].any()


# ---- refusals (CPU) ---------------------------------------------------------------

FAKE = 0x100000
FAR = {n: FAKE + 0x10000 * i for i, n in enumerate(
    "cache scales staging tok par sam n new acc out path st".split())}


def c_call(quantized=False, **over):
    a = dict(FAR, P=2, B=3, N=4, L=16, E=64, dt=1)
    a.update(over)
    p = [None if a[k] is None else ctypes.c_void_p(a[k]) for k in FAR]
    if not quantized:
        del p[1]
    lib = sv()._native.load()
    fn = lib.spec_tree_commit_quantized if quantized else lib.spec_tree_commit
    return fn(*p, a["P"], a["B"], a["N"], a["L"], a["E"], a["dt"], None)


@pytest.mark.parametrize("quantized", [False, True])
def test_host_validation(quantized):
    INVALID, UNSUP = 1, 2

    def call(**o):
        return c_call(quantized, **o)
    for name in FAR:
        if name in ("path", "st") or (name == "scales" and not quantized):
            continue
        assert call(**{name: None}) == INVALID, name
    for name in ("tok", "par", "sam", "n", "new", "acc", "out", "path", "st"):
        assert call(**{name: FAR[name] + 2}) == INVALID, name
    assert call(staging=FAR["staging"] + 1) == INVALID
    if not quantized:
        assert call(cache=FAR["cache"] + 1) == INVALID
    for o in (dict(P=-1), dict(B=-1), dict(N=0), dict(L=-1), dict(E=-1), dict(dt=7)):
        assert call(**o) == INVALID, o
    assert call(N=65) == UNSUP and call(P=1 << 20, B=1 << 20) in (INVALID, UNSUP)
    # outputs over inputs and each other
    for x in ("new", "acc", "out", "path", "st"):
        for y in ("tok", "par", "sam", "n", "new", "acc", "out", "path", "st"):
            if x == y or (x, y) in (("new", "n"), ):
                continue
            assert call(**{x: FAR[y]}) == INVALID, (x, y)
            assert call(**{x: FAR[y] + 4}) == INVALID, (x, y)
    assert call(new=FAR["n"] + 4) == INVALID
    assert call(B=0, tok=None) == 0


def test_python_refusals(monkeypatch):
    from tests.standins import Gpus, tensor
    gpus = Gpus(monkeypatch)

    def call(quantized=False, **over):
        t = dict(cache=((2, 3, 9, 64), F8 if quantized else BF), scales=((2, 3, 9, 1), E8), staging=((2, 3, 4, 64), BF),
                 tok=((3, 4), I32), par=((3, 4), I32), sam=((3, 4), I32), n=((3,), I32))
        kw = {k: over.pop(k) for k in list(over) if k in ("new_len", "status")}
        t.update(over)
        x = {k: tensor(*v) for k, v in t.items()}
        tail = (x["staging"], x["tok"], x["par"], x["sam"], x["n"])
        if quantized:
            return sv().spec_tree_commit_quantized(x["cache"], x["scales"], *tail, **kw)
        return sv().spec_tree_commit(x["cache"], *tail, **kw)
    shapes = [(3,), (3, 4), (3, 4), (3,)]
    assert [tuple(t.shape) for t in call()] == shapes and [tuple(t.shape) for t in call(True)] == shapes
    st = tensor((3,), I32)
    assert call(status=st)[3] is st
    made = len(gpus.lib.calls)
    for over in (dict(cache=((2, 3, 9, 64), torch.float16)), dict(cache=((2, 3, 9, 32), BF)), dict(cache=((2, 3), BF)),
                 dict(staging=((2, 3, 4, 64), F32)), dict(staging=((2, 2, 4, 64), BF)), dict(tok=((3, 5), I32)),
                 dict(par=((3, 4), torch.int64)), dict(sam=((4, 3), I32)), dict(n=((4,), I32)),
                 dict(new_len=tensor((3,), torch.int64)), dict(status=tensor((4,), I32))):
        with pytest.raises(ValueError):
            call(**over)
    for over in (dict(scales=((2, 3, 9, 2), E8)), dict(cache=((2, 3, 9, 64), BF)), dict(staging=((2, 3, 4, 8, 8), BF))):
        with pytest.raises(ValueError):
            call(True, **over)
    assert len(gpus.lib.calls) == made
