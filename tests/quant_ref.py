"""Plain 64-bit implementations of the 8-bit block format, the head on it and
the token log-probabilities, for the tests.  numpy, written from the
definitions: a table of the 256 e4m3 values and a nearest-value search stand
for the code, exact powers of two for the scale."""
import numpy as np
import torch

BLOCK = 128


def e4m3_table():
    """Value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = np.nan if (c & 127) == 127 else (-x if c & 128 else x)
    return v


TABLE = e4m3_table()
POSITIVE = TABLE[:127]  # ascending magnitudes, codes 0 .. 126


def encode(y):
    """Codes of |y| <= 448 (float64): the nearest value, the even code on a tie; NaN to 0x7f."""
    a = np.abs(y)
    nan = np.isnan(a)
    a = np.where(nan, 0.0, a)
    hi = np.clip(np.searchsorted(POSITIVE, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - POSITIVE[lo], POSITIVE[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.signbit(y) & ~nan, code | 128, code)
    return np.where(nan, 127, code).astype(np.uint8)


def quantize(x):
    """x [..., d] (any float array) -> (codes uint8 [..., D], scale bytes uint8 [..., nb])."""
    x = np.asarray(x, dtype=np.float64)
    d = x.shape[-1]
    nb = -(-d // BLOCK)
    v = np.zeros(x.shape[:-1] + (nb * BLOCK,))
    v[..., :d] = x
    v = v.reshape(x.shape[:-1] + (nb, BLOCK))
    finite = np.isfinite(v)
    amax = np.where(finite, np.abs(v), 0.0).max(-1)
    e = np.full(amax.shape, -126, dtype=np.int64)
    for _ in range(260):
        e += amax > 448.0 * np.exp2(e.astype(np.float64))
    y = np.where(finite, v, np.nan) / np.exp2(e.astype(np.float64))[..., None]
    return encode(y).reshape(x.shape[:-1] + (nb * BLOCK,)), (e + 127).astype(np.uint8)


def values(codes, scales, d=None):
    """float64 values of codes [..., E or D] with scale bytes [..., nb]."""
    codes = np.asarray(codes)
    step = np.exp2(np.asarray(scales, dtype=np.float64) - 127.0)
    v = TABLE[codes] * np.repeat(step, BLOCK, axis=-1)[..., :codes.shape[-1]]
    return v if d is None else v[..., :d]


def as_bytes(t):
    return t.detach().cpu().contiguous().view(torch.uint8).numpy()


def as_f64(t):
    return t.detach().cpu().double().numpy()


def same_codes(a, b):
    """Equal codes, any NaN code equal to any other, -0 told from 0."""
    a, b = np.asarray(a), np.asarray(b)
    nan = ((a & 127) == 127) & ((b & 127) == 127)
    return bool(np.all(nan | (a == b)))


def logprobs(x, token, temperature, top):
    """One row in 64 bits: (logprob, entropy, ids, top_logprobs)."""
    x = np.asarray(x, dtype=np.float64)
    V = x.shape[0]
    nan = float("nan")
    if not 0 <= token < V or np.isnan(x).any() or not np.isfinite(x.max()):
        return nan, nan, np.full(top, -1), np.full(top, nan)
    z = (x - x.max()) / temperature
    p = np.exp(z)
    lse = np.log(p.sum())
    entropy = lse - (p[p > 0] * z[p > 0]).sum() / p.sum()
    order = np.argsort(-x, kind="stable")[:top]
    order = order[x[order] > -np.inf]
    ids, lps = np.full(top, -1), np.full(top, -np.inf)
    ids[:len(order)] = order
    lps[:len(order)] = z[order] - lse
    return z[token] - lse, entropy, ids, lps
