"""Every key of a long cache counts once, in attention cut into pieces and ranges.

A row sees each entry with a score of 0 or one so far below that its weight is 0, by a pattern of its own, and entry j's
value is 1 in place j mod D.  So the weights are 1 and 0, and result d is the number of entries of the pattern at places
d mod D, over that of all of them: whole numbers below 128, and one key lost, doubled or taken with another's value
changes a numerator by one.

A result is a quotient of two sums of ones, both exact in fp32, by a reciprocal and a product: off by 3 * 2^-24 of
itself, and in bf16 by 2^-8 for its last rounding.  Of a numerator below 120 that is less than 1/2."""
import numpy as np
import pytest
import torch

from tests import tree_ref as R
from tests.test_tree_attention import BF, DEV, E8, F8, F32, sv
from tests.test_tree_plans import lengths

MOST = 120


class Counted:
    def __init__(self, B, N, Hq, Hkv, D, L, lens, share, dtype, quantized):
        self.B, self.N, self.Hq, self.Hkv, self.D, self.L, self.dtype = B, N, Hq, Hkv, D, L, dtype
        self.G = Hq // Hkv
        self.lens = [int(n) for n in lens]
        g = torch.Generator(device=DEV).manual_seed(B * L + D)
        self.parents = [-1] + [(i - 1) // 2 for i in range(1, N)]
        # Row (node i, query head h) goes by the pattern in place (i G + h) mod D of the keys.
        self.place = (torch.arange(N)[:, None] * self.G + torch.arange(Hq) % self.G) % D
        q = torch.nn.functional.one_hot(self.place, D).to(dtype).expand(B, N, Hq, D).contiguous()
        self.seen = torch.rand((B, L, Hkv, D), generator=g, device=DEV) < share
        at = (torch.arange(L, device=DEV)[:, None] + 7 * torch.arange(Hkv, device=DEV)) % D
        self.at = at
        one = torch.nn.functional.one_hot(at, D).bool().expand(B, L, Hkv, D)
        behind = (torch.arange(L, device=DEV) >= torch.tensor(self.lens, device=DEV)[:, None])[:, :, None, None]
        self.own = (torch.arange(N) * 5) % D
        new = torch.zeros((2, B, N, Hkv, D), dtype=dtype)
        new[1] = torch.nn.functional.one_hot(self.own, D).to(dtype)[None, :, None]
        tail = (*new.to(DEV), torch.tensor([self.parents] * B, dtype=torch.int32, device=DEV),
                torch.tensor(self.lens, dtype=torch.int32, device=DEV))
        if quantized:     # -448 * 4 and 1; 448 behind the sequences' ends
            k = torch.where(self.seen, 0, 0xfe).to(torch.uint8)
            v = torch.where(behind, 0x7e, torch.where(one, 0x38, 0)).to(torch.uint8)
            blocks = -(-Hkv * D // 128)
            ks, vs = (torch.full((B, L, blocks), s, dtype=torch.uint8, device=DEV) for s in (129, 127))
            self.call = lambda **kw: sv().spec_tree_attention_quantized(
                q.to(DEV), k.view(F8), ks.view(E8), v.view(F8), vs.view(E8), *tail, scale=1.0, **kw)
        else:
            k = torch.where(self.seen, 0.0, -1000.0).to(dtype)
            v = torch.where(behind, 448.0, one.to(dtype)).to(dtype)
            self.call = lambda **kw: sv().spec_tree_attention(q.to(DEV), k, v, *tail, scale=1.0, **kw)

    def counts(self, b, h, window, sinks):
        """[N, G, D] numerators and [N, G, 1] denominators of a sequence's KV head."""
        n, D = self.lens[b], self.D
        nodes = R.lines(self.parents)
        num = np.zeros((self.N, self.G, D))
        all_j = torch.arange(n, device=DEV)
        whole = None
        for i, line in enumerate(nodes):
            if window or whole is None:
                sees = (all_j < sinks) | (all_j > n + len(line) - 1 - window) if window else all_j >= 0
                j = all_j[sees]
                whole = torch.zeros((D, D), device=DEV).index_add_(0, self.at[j, h], self.seen[b, j, h].float())
                whole = whole.T.cpu().numpy()     # by pattern, then place of the value
            num[i] = whole[self.place[i, :self.G].numpy()]
            for a in line:
                position = n + len(nodes[a]) - 1
                if not window or position < sinks or position > n + len(line) - 1 - window:
                    num[i, :, self.own[a]] += 1
        return num, num.sum(-1, keepdims=True)

    def check(self, window=0, sinks=0):
        got = self.call(window=window, sinks=sinks).double().cpu().numpy()
        off = 4 * 2.0 ** -24 + (2.0 ** -8 if self.dtype is BF else 0)
        for b in range(self.B):
            for h in range(self.Hkv):
                num, den = self.counts(b, h, window, sinks)
                assert num.max() < MOST and MOST * off < 0.5
                here = got[b, :, h * self.G:(h + 1) * self.G]
                bad = np.abs(here * den - num) > num * off
                assert not bad.any(), (b, h, np.argwhere(bad)[:8], (here * den)[bad][:8], num[bad][:8])


FORMS = {
    "pieces": dict(B=1, N=4, Hq=4, Hkv=1, D=128, L=20011, lens=[20000], share=0.5),
    "pieces of heads of 64": dict(B=1, N=4, Hq=4, Hkv=1, D=64, L=20011, lens=[19999], share=0.25),
    "pieces of heads of 72": dict(B=1, N=7, Hq=4, Hkv=1, D=72, L=20011, lens=[20011], share=0.25),
    "pieces of heads of 256": dict(B=1, N=5, Hq=4, Hkv=1, D=256, L=30011, lens=[30000], share=0.5),
    "pieces of two heads": dict(B=2, N=9, Hq=4, Hkv=2, D=128, L=9001, lens=[9001, 4567], share=0.5),
    "pieces of shared keys": dict(B=1, N=40, Hq=4, Hkv=1, D=128, L=16400, lens=[16383], share=0.5),
    "pieces of shared keys of 64": dict(B=2, N=64, Hq=4, Hkv=1, D=64, L=9001, lens=[8990, 77], share=0.5),
    "one block a pair": dict(B=3, N=6, Hq=6, Hkv=3, D=64, L=1000, lens=[1000, 999, 31], share=1.0),
    "ranges": dict(B=260, N=2, Hq=4, Hkv=1, D=64, L=2100, lens=lengths(260, 2100, {0: 2100, 99: 1500, 259: 2099}, 3),
                   share=0.5),
    "ranges, one long sequence": dict(B=64, N=2, Hq=4, Hkv=1, D=64, L=20000, lens=lengths(64, 20000, {41: 20000}, 4),
                                      share=0.25),
    "ranges of many rows": dict(B=64, N=64, Hq=8, Hkv=2, D=64, L=9000,
                                lens=lengths(64, 9000, {b: 137 * b + 300 for b in range(0, 64, 3)}, 5), share=0.5),
}


@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("form", sorted(FORMS))
def test_every_key_counts_once(form, dtype, quantized):
    Counted(dtype=dtype, quantized=quantized, **FORMS[form]).check()


@pytest.mark.gpu
@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("form", ["pieces", "pieces of two heads", "pieces of shared keys", "ranges"])
@pytest.mark.parametrize("window,sinks", [(1700, 130), (5000, 0)])
def test_every_key_of_a_window_counts_once(form, dtype, quantized, window, sinks):
    Counted(dtype=dtype, quantized=quantized, **FORMS[form]).check(window, sinks)


@pytest.mark.parametrize("lost", [1, 16, 32, 64])
def test_lost_and_doubled_keys_would_show(lost):
    """On the oracle: a run of keys left out or taken twice moves a numerator by more than the bound of both."""
    D, n, line = 128, 20000, 3
    seen = np.random.default_rng(0).random(n) < 0.5
    off = 4 * 2.0 ** -24 + 2.0 ** -8

    def count(keys):
        num = np.bincount(keys % D, minlength=D).astype(float)
        num[:line] += 1
        return num
    keys = np.flatnonzero(seen)
    num = count(keys)
    den = num.sum()
    for first in (0, 31, 5000, n - lost):
        run = keys[(keys >= first) & (keys < first + lost)]
        if not len(run):
            continue
        for other in (np.setdiff1d(keys, run), np.sort(np.concatenate([keys, run]))):
            got = count(other) / count(other).sum()
            assert (np.abs(got * den - num) * (1 - 2.0 ** -8) > num * off).any()
