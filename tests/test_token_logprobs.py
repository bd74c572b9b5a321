"""Token log-probabilities, entropies and alternatives against 64-bit rows.

Ids of alternatives are compared for equality (the order is by the logits as
they are).  Tolerance of the logarithms: an exponential is off by one step of
the instruction and half a step of its argument (|t| <= 20 carries weight),
a tile's fp32 sums by 16 additions in a lane, 2 across its chains and 6 across
lanes, so Z is off by at most (2 + 20 + 24) half steps, and H by as many of
its magnitude; log2(e) / T and the result are rounded once each, relative to
the value: 2^-24 * (64 + 4 |value|) covers them."""
import ctypes

import numpy as np
import pytest
import torch

from tests import quant_ref as R

DEV = torch.device("cuda", 0)
BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


def sv():
    import speculative_sampling_verification_vocab_amd as m
    return m


def close(got, want):
    got, want = np.asarray(got, dtype=np.float64), np.asarray(want, dtype=np.float64)
    # a result past the largest float32 plus half its step, 2^128 - 2^103, rounds to infinity
    want = np.where(np.abs(want) >= 2.0 ** 128 - 2.0 ** 103, np.copysign(INF, want), want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), (got, want)
    assert np.array_equal(np.isinf(got), np.isinf(want)), (got, want)
    f = np.isfinite(want)
    tol = 2.0 ** -24 * (64 + 4 * np.abs(want[f]))
    assert np.all(np.abs(got[f] - want[f]) <= tol), (np.max(np.abs(got[f] - want[f]) / tol), got[f], want[f])


def check(x, tokens, top, T=1.0):
    """x [N, V] on the CPU, of the type under test."""
    T = float(np.float32(T))
    t = torch.as_tensor(np.asarray(tokens), dtype=torch.int32)
    got = [g.cpu().numpy() for g in sv().spec_token_logprobs(x.to(DEV), t.to(DEV), top, T)]
    compare(x, t, top, T, got)
    return got


def compare(x, t, top, T, got):
    N = x.shape[0]
    assert got[0].shape == got[1].shape == (N,) and got[2].shape == got[3].shape == (N, top)
    for i in range(N):
        lp, ent, ids, lps = R.logprobs(R.as_f64(x[i]), int(t[i]), T, top)
        assert np.array_equal(got[2][i], ids), (i, got[2][i], ids)
        close(got[0][i], lp)
        close(got[1][i], ent)
        close(got[3][i], lps)


def normal(N, V, dtype, seed, std=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(N, V, generator=g) * std).to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [1, 2, 7, 31, 33, 500, 512, 513, 1023, 4096, 4097, 5003, 8200, 32000, 50001, 128256])
def test_vocabularies(V, dtype):
    """From one token up, odd lengths (rows that begin anywhere on the 16-byte grid) among them."""
    print(f"case V={V} {dtype}", flush=True)
    N = 9
    x = normal(N, V, dtype, V)
    tokens = torch.randint(0, V, (N,), generator=torch.Generator().manual_seed(V + 1)).numpy()
    tokens[0], tokens[1] = V - 1, 0
    tokens[4], tokens[5] = -1, V
    check(x, tokens, 20)


@pytest.mark.gpu
@pytest.mark.parametrize("top", [0, 1, 2, 5, 31, 32])
def test_alternatives(top):
    check(normal(5, 20001, BF, 11), [3, 20000, -1, 77, 4096], top)
    check(normal(3, 40, F32, 12), [39, 0, 5], top)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,V", [(BF, 262144), (BF, 600003), (F32, 300001)])
def test_large_vocabularies(dtype, V):
    """The largest benchmarked vocabulary, and more chunks than the pick keeps in LDS."""
    check(normal(3, V, dtype, 5), [V - 1, 1, 1000], 32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_ties(dtype):
    V = 9001
    g = torch.Generator().manual_seed(9)
    x = torch.zeros(8, V)
    x[1] = torch.randint(0, 2, (V,), generator=g).float()          # two values
    x[2] = torch.randint(0, 40, (V,), generator=g).float() / 8     # few values
    x[3] = torch.arange(V).float() / 64                            # ascending (ties in bf16)
    x[4] = -torch.arange(V).float() / 64                           # descending
    x[5, ::2] = -0.0                                               # -0 ties with 0
    x[6] = torch.sort(torch.randn(V, generator=g))[0]
    x[7, 4090:4110] = 1.0                                          # across a tile's border
    check(x.to(dtype), [0, 1, 2, 9000, 4, 5, 6, 4100], 32)
    check(x.to(dtype)[:, :300].contiguous(), [0, 1, 2, 299, 4, 5, 6, 7], 32)   # fewer chunks than alternatives


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_masked_rows(dtype):
    V = 10007
    g = torch.Generator().manual_seed(10)
    x = torch.randn(12, V, generator=g) * 3
    x[0, torch.rand(V, generator=g) < 0.5] = -INF
    x[1] = -INF                                     # nothing left: no law
    x[2] = -INF
    x[2, 7777] = 2.0                                # one token left
    x[3] = -INF
    x[3, [5, 4096, 9999]] = torch.tensor([1.0, 3.0, 1.0])
    x[4, :8192] = -INF                              # whole tiles masked
    x[5, 100] = NAN
    x[6, 9000] = INF
    x[7] = torch.finfo(dtype).min                   # the type's lowest value as a mask ..
    x[7, :10] = torch.arange(10).float()
    x[8] = torch.finfo(dtype).min                   # .. and nothing else
    x[9, torch.rand(V, generator=g) < 0.9] = torch.finfo(dtype).min
    x[10, 3] = -INF                                 # the token itself
    x[11] = -INF
    x[11, 1000:1200] = torch.randn(200, generator=g)
    check(x.to(dtype), [1, 1, 7777, 5, 9000, 1, 1, 3, 8, 4, 3, 1100], 20)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [500, 40003, 300001])
def test_tokens_far_below_the_rest(V, dtype):
    """A token's own logit is no reference for its row: the lowest value, -inf, far below, at a low temperature."""
    x = normal(6, V, dtype, 22)
    x[0, 7] = torch.finfo(dtype).min
    x[1, 7] = -INF
    x[2, 7] = -1.0e4
    x[3, 7] = -60.0
    x[4, :] = -50.0
    x[4, V - 1] = 10.0
    x[5, :V // 2] = torch.finfo(dtype).min
    for T in (1.0, 0.01, 100.0):
        check(x, [7, 7, 7, 7, 7, 7], 12, T)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [9001, 66000, 300001])
def test_many_equal_rows_at_once(V, dtype):
    """Rows that fall back to one chunk after another, on every CU at once, among ordinary ones."""
    N = 600
    x = normal(N, V, dtype, 23)
    x[::2] = 1.5
    x[1::4, 100:5000] = 20.0
    t = torch.arange(N, dtype=torch.int32) % V
    got = [v.cpu().numpy() for v in sv().spec_token_logprobs(x.to(DEV), t.to(DEV), 20)]
    some = [0, 1, 2, 3, 5, 301, 598, 599]
    compare(x[some], t[some], 20, 1.0, [v[some] for v in got])
    assert (got[2][::2] == np.arange(20)).all()
    assert (got[2][1::4] == np.arange(100, 120)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,V", [(3, 40000), (3, 300001), (300, 40003)])
def test_masked_before_a_fault(N, V, dtype):
    """-inf in the first tiles and a NaN or +inf in a later one, in each form of the launch."""
    x = normal(3, V, dtype, 21)
    x[:, :9000] = -INF
    x[0, V - 5], x[1, V - 3] = NAN, INF
    x = x.repeat(N // 3, 1)
    t = torch.full((N,), V - 1, dtype=torch.int32)
    got = [g.cpu().numpy() for g in sv().spec_token_logprobs(x.to(DEV), t.to(DEV), 7)]
    compare(x[:3], t[:3], 7, 1.0, [g[:3] for g in got])
    # the others hold the same rows, at other alignments where V is odd: sums are then grouped otherwise
    for i in range(3, N, 31):
        compare(x[i:i + 1], t[i:i + 1], 7, 1.0, [g[i:i + 1] for g in got])


@pytest.mark.gpu
@pytest.mark.parametrize("N,V,dtype", [(257, 40003, BF), (257, 66000, F32), (40, 140000, BF), (700, 20000, BF),
                                       (2050, 3001, F32)])
def test_batches(N, V, dtype):
    """Each form of the launch, odd and even rows, dead ones among them."""
    g = torch.Generator().manual_seed(N)
    x = normal(7, V, dtype, V).repeat(N // 7 + 1, 1)[:N].contiguous()
    t = torch.randint(-1, V + 1, (N,), generator=g).to(torch.int32)
    t[::3] = -1
    got = [v.cpu().numpy() for v in sv().spec_token_logprobs(x.to(DEV), t.to(DEV), 12)]
    some = torch.randperm(N, generator=g)[:25]
    compare(x[some], t[some], 12, 1.0, [v[some.numpy()] for v in got])
    assert np.array_equal(np.isnan(got[0]), ((t < 0) | (t >= V)).numpy())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1.2e-38, 1e-30, 1e-8, 1e-3, 0.3, 2.0, 1e4, 1e30, 3e38])
def test_temperatures(T, dtype):
    check(normal(4, 5001, dtype, 13), [0, 5000, 17, 300], 8, T)


@pytest.mark.gpu
def test_large_logits():
    for scale in (1e10, 1e30, 1e37):
        check(normal(3, 5001, F32, 14) * scale, [0, 5000, 17], 8)
        check(normal(3, 5001, F32, 15) * scale, [0, 5000, 17], 8, scale)


@pytest.mark.gpu
def test_sharp_and_flat_rows():
    x = torch.zeros(3, 70000)
    x[0, 12345] = 30.0                              # entropy and log-probability near zero
    x[1] = -100.0
    x[1, 5] = 0.0
    check(x.to(BF), [12345, 5, 3], 3)


@pytest.mark.gpu
def test_rows_off_their_alignment():
    for dtype in (BF, F32):
        flat = normal(1, 3 * 6000 + 1, dtype, 16)[0].to(DEV)
        x = flat[1:].view(3, 6000)
        t = torch.tensor([5, 5999, 0], dtype=torch.int32)
        got = [g.cpu().numpy() for g in sv().spec_token_logprobs(x, t.to(DEV), 9)]
        compare(x.cpu(), t, 9, 1.0, got)


@pytest.mark.gpu
def test_dead_rows_are_not_read():
    """Rows without a token may hold anything; their outputs are NaN and -1."""
    x = normal(6, 3001, BF, 17)
    x[1::2] = NAN
    got = check(x, [4, -1, 5, 3001, 6, -2147483648], 4)
    assert np.isnan(got[0][1::2]).all() and (got[2][1::2] == -1).all()


@pytest.mark.gpu
def test_same_on_every_call():
    x = normal(40, 30011, BF, 18).to(DEV)
    t = torch.arange(40, dtype=torch.int32, device=DEV)
    a = sv().spec_token_logprobs(x, t, 20)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(a, sv().spec_token_logprobs(x, t, 20)))
    one = [sv().spec_token_logprobs(x[i:i + 1].contiguous(), t[i:i + 1], 20) for i in range(0, 40, 13)]
    for k, i in enumerate(range(0, 40, 13)):       # nor do they depend on the batch
        if (i * 30011 * 2) % 16 == 0:
            assert all(torch.equal(p[0], q[i]) for p, q in zip(one[k], a))


@pytest.mark.gpu
def test_empty_and_leading_dims():
    e = sv().spec_token_logprobs(torch.empty(0, 100, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV), 3)
    assert [tuple(v.shape) for v in e] == [(0,), (0,), (0, 3), (0, 3)]
    x = normal(6, 333, F32, 19)
    t = torch.arange(6, dtype=torch.int32)
    a = sv().spec_token_logprobs(x.view(2, 3, 333).to(DEV), t.view(2, 3).to(DEV), 3)
    assert a[0].shape == (2, 3) and a[2].shape == (2, 3, 3)
    compare(x, t, 3, 1.0, [v.flatten(0, 1).cpu().numpy() for v in a])
    one = sv().spec_token_logprobs(x[0].to(DEV), t[0].to(DEV), 3)
    assert one[0].shape == () and torch.equal(one[2], a[2][0, 0])


# ---- refusals -----------------------------------------------------------------------

OK, INVALID, UNSUP, WS = 0, 1, 2, 3


def test_refusals():
    from speculative_sampling_verification_vocab_amd import _native
    lib, p = _native.load(), ctypes.c_void_p
    size = lib.spec_token_logprobs_workspace_bytes
    ok = dict(x=0x10000, t=0x20000, N=4, V=1000, dt=1, T=1.0, top=5, lp=0x30000, ent=0x40000, ids=0x50000,
              tl=0x60000, ws=0x100000, wb=1 << 30)

    def call(**o):
        a = {**ok, **o}
        return lib.spec_token_logprobs(p(a["x"]), p(a["t"]), a["N"], a["V"], a["dt"], ctypes.c_float(a["T"]), a["top"],
                                       p(a["lp"]), p(a["ent"]), p(a["ids"]), p(a["tl"]), p(a["ws"]), a["wb"], None)
    for name in ("x", "t", "lp", "ids", "tl"):
        assert call(**{name: None}) == INVALID, name
    for name in ("t", "lp", "ent", "ids", "tl"):
        assert call(**{name: 0x70002}) == INVALID, name
    assert call(x=0x10001) == INVALID and call(x=0x10002, dt=0) == INVALID
    assert call(N=-1) == INVALID and call(V=0) == INVALID and call(dt=3) == INVALID and call(top=-1) == INVALID
    for T in (0.0, -1.0, NAN, INF, 1e-39):
        assert call(T=T) == INVALID, T
    assert call(top=33) == UNSUP and call(V=(1 << 30) + 1) == UNSUP
    assert call(N=0x7fffffff, V=1 << 20) == UNSUP
    need = size(4, 200000, 1, 5)
    assert need > size(4, 200000, 1, 0) > 0
    for o in (dict(ws=None), dict(ws=0x100080), dict(wb=need - 1)):
        assert call(V=200000, **o) == WS
    assert size(4, 1000, 1, 5) == 0                       # short rows need none
    assert call(N=0, x=None, ws=None) == OK
    assert size(0, 1000, 1, 5) == 0 and size(4, 0, 1, 5) == 0 and size(4, 1000, 1, 33) == 0


def test_cpu_tensors_are_refused():
    with pytest.raises(ValueError):
        sv().spec_token_logprobs(torch.zeros(2, 10), torch.zeros(2, dtype=torch.int32))


@pytest.mark.gpu
def test_shapes_and_types_are_checked():
    x, t = torch.zeros(4, 64, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
    f = sv().spec_token_logprobs
    for a in ((x.half(), t), (x, t.long()), (x, t[:3]), (x, t.cpu()), (x.t(), t), (x, t, -1)):
        with pytest.raises(ValueError):
            f(*a)
    with pytest.raises(sv().SpecVerifyError):
        f(x, t, 33)
    for T in (0.0, -1.0, NAN, INF):
        with pytest.raises(sv().SpecVerifyError):
            f(x, t, 2, T)
