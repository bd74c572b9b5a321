"""Tokens drawn with request settings, against a plain draw in long double.

The weights of the law are whole multiples of 2^-F of the largest one, F = 62 - ceil(log2 V), at most 50, and
exact to 2^-46 of themselves beside that (an exponential whose argument, up to 64 in size, is rounded to 2^-53 of
itself).  So a sum of up to V of them, of a total of at most V, and the uniform's or share's product with the
total, are off by less than V (2^-F + 2^-45) of the largest weight.  The plain draw says how far its nearest
border is from the uniform; beyond twice that bound, the token has to be the same."""
import ctypes
import math

import numpy as np
import pytest
import torch

from tests import tree_ref as R

DEV = torch.device("cuda", 0)
BF, F32 = torch.bfloat16, torch.float32
OFF = (1.0, 0, 1.0, 0.0)


def sv():
    import speculative_sampling_verification_vocab_amd as m
    return m


def near(V):
    F = min(50, 62 - math.ceil(math.log2(V)) if V > 1 else 62)
    return 2 * V * (2.0 ** -F + 2.0 ** -45)


def check(x, u, settings, got=None):
    """x [R, V] on the CPU, u [R], settings: four numbers, or four lists of R."""
    R_, V = x.shape
    rows = [v if isinstance(v, (list, tuple)) else [v] * R_ for v in settings]
    if got is None:
        arg = []
        for v, t in zip(settings, (F32, torch.int32, F32, F32)):
            arg.append(torch.tensor(v, dtype=t, device=DEV) if isinstance(v, (list, tuple)) else v)
        got = sv().spec_sample_tokens(x.to(DEV), torch.as_tensor(u, dtype=F32).to(DEV), arg[0], top_k=arg[1],
                                      top_p=arg[2], min_p=arg[3])
    got = got.cpu().tolist()
    xs = x.double().numpy()
    close = 0
    for r in range(R_):
        want, margin = R.sample(xs[r], u[r], rows[0][r], rows[1][r], rows[2][r], rows[3][r])
        if margin <= near(V):
            close += 1
            continue
        assert got[r] == want, (r, got[r], want, [v[r] for v in rows], float(u[r]), margin)
    return close


def logits(rows, V, dtype, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((rows, V), generator=g) * spread).to(dtype), torch.rand(rows, generator=g).tolist()


SETTINGS = [OFF, (0.75, 50, 1.0, 0.0), (1.0, 0, 0.9, 0.0), (0.6, 40, 0.9, 0.0), (1.0, 0, 1.0, 0.05), (0.0, 0, 1.0, 0.0),
            (1.3, 200, 0.97, 0.03), (1.5, 0, 0.99, 0.01), (1.0, 1, 1.0, 0.0), (1.0, 5, 0.5, 0.5), (0.1, 1000, 0.95, 0.0),
            (4.0, 0, 0.999, 0.0), (1.0, 0, 1e-6, 0.0), (2.0, 2, 1.0, 0.0), (1.0, 1500, 0.9, 0.0), (3.0, 5000, 1.0, 0.0)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 9, 63, 255, 511, 512, 513, 1000, 4095, 8192, 8193, 50257])
def test_settings_over_row_lengths(dtype, V):
    x, u = logits(2 * len(SETTINGS), V, dtype, V)
    assert check(x, u, tuple(list(c) for c in zip(*(SETTINGS * 2)))) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [128256, 262144, 300001])
def test_large_vocabularies(dtype, V):
    x, u = logits(len(SETTINGS), V, dtype, V)
    x -= torch.log(torch.arange(1, V + 1)).to(dtype)
    assert check(x, u, tuple(list(c) for c in zip(*SETTINGS))) <= 1


@pytest.mark.gpu
def test_a_vocabulary_of_two_million():
    """Rows of more than 2^20 tokens: chunks of several hundred tokens."""
    V = 2_000_003
    x, u = logits(4, V, BF, 1, spread=1.0)
    check(x, u, ([1.0, 1.0, 1.0, 0.0], [0, 3000, 0, 0], [1.0, 1.0, 0.5, 1.0], [0.0, 0.0, 0.0, 0.0]))


@pytest.mark.gpu
@pytest.mark.parametrize("settings", SETTINGS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_setting_for_all_rows(settings, dtype):
    x, u = logits(24, 3001, dtype, 5)
    assert check(x, u, settings) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [1, 5, 700, 40000])
def test_equal_logits(dtype, V):
    """All alike, and of few values: cuts fall inside ties, which go by the lower id."""
    g = torch.Generator().manual_seed(V)
    x = torch.full((12, V), 2.5, dtype=dtype)
    x[6:] = torch.randint(0, 3, (6, V), generator=g).to(dtype)
    u = [0.0, 0.3, 0.999999] * 4
    for s in (OFF, (1.0, 3, 1.0, 0.0), (1.0, 0, 0.3, 0.0), (1.0, 600, 0.77, 0.0), (0.5, 0, 1.0, 0.9), (0.0, 0, 1.0, 0.0)):
        check(x, u, s)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [2, 4, 64])
def test_shares_that_ties_reach_exactly(n):
    """n equal tokens: a top-p of 1/2 keeps exactly half of them, whose weights reach it; the next
    float above keeps one more.  u picks the last kept one."""
    x = torch.full((3, n), -1.25, dtype=F32)
    half = np.float32(0.5)
    p = [float(half), float(np.nextafter(half, np.float32(1))), float(np.nextafter(half, np.float32(0)))]
    got = sv().spec_sample_tokens(x.to(DEV), torch.full((3,), 0.99999, device=DEV), top_p=torch.tensor(p, device=DEV))
    assert got.tolist() == [n // 2 - 1, n // 2, n // 2 - 1]


@pytest.mark.gpu
def test_borders_of_equal_tokens():
    """u = i / 8 of eight equal tokens is token i's: the cumulative weight has to exceed u."""
    u = [i / 8 for i in range(8)] + [float(np.nextafter(np.float32(i / 8), np.float32(0))) for i in range(1, 8)]
    got = sv().spec_sample_tokens(torch.zeros((15, 8), device=DEV), torch.tensor(u, device=DEV))
    assert got.tolist() == list(range(8)) + list(range(7))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_masked_tokens_are_never_drawn(dtype):
    """-inf and the type's lowest value, in front, behind and between; rows with one token left."""
    for low in (-float("inf"), torch.finfo(dtype).min):
        x, u = logits(32, 900, dtype, 3)
        g = torch.Generator().manual_seed(4)
        x[torch.rand(x.shape, generator=g) < 0.7] = low
        x[0, 1:] = low
        x[1, :-1] = low
        x[2, :450] = low
        u[0], u[1], u[2], u[3] = 0.0, 0.9999999, 0.0, 0.0
        for s in ((1.0, 0, 1.0, 0.0), (1.0, 800, 1.0, 0.0), (1.0, 0, 0.99, 0.0), (2.0, 500, 0.999, 1e-30)):
            assert check(x, u, s) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_zeros_of_both_signs_are_equal(dtype):
    x = torch.tensor([[-0.0, 0.0, -0.0, 0.0, -5.0]]).to(dtype).expand(4, 5).contiguous()
    got = sv().spec_sample_tokens(x.to(DEV), torch.tensor([0.0, 0.6, 0.4, 0.9], device=DEV),
                                  torch.tensor([0.0, 1.0, 1.0, 1.0], device=DEV),
                                  top_k=torch.tensor([0, 2, 3, 1], dtype=torch.int32, device=DEV))
    assert got.tolist() == [0, 1, 1, 0]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_extreme_temperatures_and_values(dtype):
    x, u = logits(8, 500, dtype, 6)
    big = torch.tensor(torch.finfo(dtype).max)
    for T in (1e-45, 1e-30, 1e-3, 1e4, 1e30, 3e38):
        check(x, u, (T, 0, 0.9, 0.0))
        check((x / x.abs().max() * big).to(dtype), u, (T, 30, 1.0, 0.2))
    x[:, 3] = big.to(dtype)
    x[:, 4] = -big.to(dtype)
    check(x, u, (1.0, 0, 1.0, 0.0))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_faulty_rows(dtype):
    nan, inf = float("nan"), float("inf")
    x, u = logits(16, 2000, dtype, 7)
    x[0, 77] = nan
    x[1, 1999] = inf
    x[2] = -inf
    x[3, 0] = -nan
    x[4] = nan
    T, k, p, m = [1.0] * 16, [0] * 16, [1.0] * 16, [0.0] * 16
    T[5], T[6], T[7] = nan, -1.0, inf
    p[8], m[9] = nan, nan
    u[10], u[11], u[12] = nan, 1.0, -0.5
    T[13], x[13, 5] = 0.0, nan
    got = sv().spec_sample_tokens(x.to(DEV), torch.tensor(u, device=DEV), torch.tensor(T, device=DEV),
                                  top_k=torch.tensor(k, dtype=torch.int32, device=DEV), top_p=torch.tensor(p, device=DEV),
                                  min_p=torch.tensor(m, device=DEV))
    assert got[:14].tolist() == [-1] * 14 and (got[14:] >= 0).all()
    check(x[14:], u[14:], OFF, got[14:])


@pytest.mark.gpu
def test_settings_that_are_off():
    """Values of top_k, top_p and min_p that mean "all tokens", and those that leave one."""
    x, u = logits(10, 1500, F32, 8)
    got = [sv().spec_sample_tokens(x.to(DEV), torch.tensor(u, device=DEV), top_k=k, top_p=p, min_p=m).tolist()
           for k, p, m in ((0, 1.0, 0.0), (-5, 2.0, -1.0), (1500, 1.0, 0.0), (2 ** 31 - 1, float("inf"), -float("inf")))]
    assert all(g == got[0] for g in got)
    best = x.argmax(-1).tolist()
    for k, p, m in ((1, 1.0, 0.0), (0, 0.0, 0.0), (0, -3.0, 0.0), (0, 1.0, 1.0), (0, 1.0, 7.0)):
        assert sv().spec_sample_tokens(x.to(DEV), torch.tensor(u, device=DEV), top_k=k, top_p=p,
                                       min_p=m).tolist() == best


@pytest.mark.gpu
def test_many_draws_follow_the_law():
    """2^16 uniforms, one in each of 2^16 equal steps: each token's count is within 2 of its probability's."""
    x, _ = logits(1, 40, F32, 9, spread=1.0)
    n = 1 << 16
    u = (torch.arange(n, dtype=torch.float64) + 0.5) / n
    got = sv().spec_sample_tokens(x.expand(n, 40).contiguous().to(DEV), u.float().to(DEV), 0.8, top_k=25, top_p=0.9)
    w = np.exp((x[0].double().numpy() - x.max().item()) / np.float32(0.8))
    order = np.argsort(-w)
    mass = np.cumsum(w[order][:25])
    keep = order[:int(np.searchsorted(mass, np.float32(0.9) * mass[-1])) + 1]
    law = np.zeros(40)
    law[keep] = w[keep] / w[keep].sum()
    assert np.abs(np.bincount(got.cpu().numpy(), minlength=40) - n * law).max() <= 2


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_of_any_alignment_and_leading_dimensions(dtype):
    x, u = logits(12, 1237, dtype, 10)
    base = torch.zeros(12 * 1237 + 3, dtype=dtype, device=DEV)
    base[3:] = x.flatten().to(DEV)
    view = base[3:].view(3, 4, 1237)
    got = sv().spec_sample_tokens(view, torch.tensor(u, device=DEV).view(3, 4), 0.9, top_k=70, top_p=0.95)
    assert got.shape == (3, 4) and got.dtype is torch.int32
    check(x, u, (0.9, 70, 0.95, 0.0), got.flatten())
    one = sv().spec_sample_tokens(view[0, 0], torch.tensor(u[0], device=DEV), 0.9, top_k=70, top_p=0.95)
    assert one.shape == () and int(one) == int(got[0, 0])


@pytest.mark.gpu
def test_only_the_tokens_are_written_and_always_the_same():
    x, u = logits(700, 4000, BF, 11)
    xd, ud = x.to(DEV), torch.tensor(u, device=DEV)
    guard = torch.full((1000,), 99, dtype=torch.int32, device=DEV)
    out = guard[100:800]
    first = sv().spec_sample_tokens(xd, ud, 1.1, top_p=0.9, out=out)
    assert first is out and (guard[:100] == 99).all() and (guard[800:] == 99).all()
    assert torch.equal(xd.cpu(), x)
    for _ in range(3):
        assert torch.equal(sv().spec_sample_tokens(xd, ud, 1.1, top_p=0.9), first)


@pytest.mark.gpu
def test_rows_beyond_2_to_the_32_values():
    V = 1 << 20
    R_ = (1 << 12) + 2
    x = torch.zeros((R_, V), dtype=BF, device=DEV)
    x[-1, 12345], x[-2, 7] = 30.0, 30.0
    u = torch.full((R_,), 0.5, device=DEV)
    got = sv().spec_sample_tokens(x, u, 1.0, top_k=1)
    assert got[-1].item() == 12345 and got[-2].item() == 7 and not got[:-2].any()


def test_empty_call(monkeypatch):
    from tests.standins import Gpus, tensor
    gpus = Gpus(monkeypatch)
    assert sv().spec_sample_tokens(tensor((0, 9), BF), tensor((0,), F32)).shape == (0,)
    assert len(gpus.lib.calls) == 1


# ---- refusals (CPU) ---------------------------------------------------------------

FAKE = 0x10000


def c_call(**over):
    a = dict(x=FAKE, u=FAKE, R=2, V=100, dt=1, T=None, aT=1.0, k=None, ak=0, p=None, ap=1.0, m=None, am=0.0, out=FAKE)
    a.update(over)
    q = {k: ctypes.c_void_p(v) if k in ("x", "u", "T", "k", "p", "m", "out") and v is not None else v for k, v in a.items()}
    f = ctypes.c_float
    return sv()._native.load().spec_sample_tokens(q["x"], q["u"], a["R"], a["V"], a["dt"], q["T"], f(a["aT"]), q["k"],
                                                  a["ak"], q["p"], f(a["ap"]), q["m"], f(a["am"]), q["out"], None)


def test_host_validation():
    INVALID, UNSUP = 1, 2
    nan = float("nan")
    for o in (dict(x=None), dict(u=None), dict(out=None), dict(R=-1), dict(V=0), dict(dt=3), dict(aT=-0.5), dict(aT=nan),
              dict(aT=float("inf")), dict(ap=nan), dict(am=nan), dict(x=FAKE + 1), dict(u=FAKE + 2), dict(out=FAKE + 1),
              dict(T=FAKE + 1), dict(k=FAKE + 2), dict(p=FAKE + 3), dict(m=FAKE + 1)):
        assert c_call(**o) == INVALID, o
    assert c_call(V=(1 << 30) + 1) == UNSUP and c_call(R=0x7fffffff) == UNSUP
    assert c_call(R=0, x=None, u=None, out=None) == 0


def test_python_refusals(monkeypatch):
    from tests.standins import Gpus, tensor
    gpus = Gpus(monkeypatch)
    x, u = tensor((2, 9), BF), tensor((2,), F32)
    I32 = torch.int32
    assert sv().spec_sample_tokens(x, u, tensor((2,), F32), top_k=tensor((2,), I32)).shape == (2,)
    for a, kw in (((tensor((2, 9), torch.float16), u), {}), ((tensor((), BF), u), {}), ((tensor((2, 0), BF), u), {}),
                  ((x, tensor((3,), F32)), {}), ((x, tensor((2,), BF)), {}), ((x, u, tensor((2, 1), F32)), {}),
                  ((x, u, tensor((2,), BF)), {}), ((x, u), dict(top_k=tensor((2,), torch.int64))),
                  ((x, u), dict(top_p=tensor((1,), F32))), ((x, u), dict(min_p=tensor((2,), I32))),
                  ((x, u), dict(out=tensor((2,), torch.int64))), ((x, u), dict(out=tensor((3,), I32)))):
        with pytest.raises(ValueError):
            sv().spec_sample_tokens(*a, **kw)
    assert len(gpus.lib.calls) == 1
    with pytest.raises(ValueError):   # no CPU path
        sv().spec_sample_tokens(torch.zeros(2, 9), torch.zeros(2))
