"""Plain implementations of the operators of a step with a tree of drafts, for
the tests: attention in 64 bits entry by entry, draws in numpy's long double,
the walk as a loop.  Written from the definitions."""
import numpy as np


def lines(parents):
    """For each node the list from its first ancestor to itself, or None for an absent one."""
    out = []
    for i, p in enumerate(parents):
        if p == -1:
            out.append([i])
        elif 0 <= p < i and out[p] is not None:
            out.append(out[p] + [i])
        else:
            out.append(None)
    return out


def attention(q, k_cache, v_cache, k_new, v_new, parents, cache_len, scale, window=0, sinks=0):
    """float64 arrays as spec_tree_attention takes them.  Returns (out, spread, score): out [B, N, Hq, D];
    spread, the weighted mean of |v|, of out's shape, and score, the largest sum of |q||k| * scale of a
    row [B, N, Hq, 1], which rounding errors go by."""
    B, N, Hq, D = q.shape
    L, Hkv = k_cache.shape[1], k_cache.shape[2]
    out, spread, score = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, N, Hq, 1))
    for b in range(B):
        n = int(cache_len[b])
        if not 0 <= n <= L:
            out[b] = np.nan
            continue
        for i, line in enumerate(lines([int(p) for p in parents[b]])):
            if line is None:
                continue
            at = n + len(line) - 1
            places = list(range(n)) + [n + d for d in range(len(line))]
            sees = [t for t, p in enumerate(places) if not window or p < sinks or p > at - window]
            for h in range(Hq):
                g = h // (Hq // Hkv)
                k = np.concatenate([k_cache[b, :n, g], k_new[b, line, g]])[sees]
                v = np.concatenate([v_cache[b, :n, g], v_new[b, line, g]])[sees]
                with np.errstate(invalid="ignore", over="ignore"):
                    x = k @ q[b, i, h] * scale
                    score[b, i, h] = np.max(np.abs(k) @ np.abs(q[b, i, h])) * scale
                    if np.all(x == -np.inf):
                        continue
                    p = np.exp(x - np.max(x))
                    out[b, i, h] = (p[:, None] * v).sum(0) / p.sum()
                    spread[b, i, h] = (p[:, None] * np.abs(v)).sum(0) / p.sum()
    return out, spread, score


def attention_bound(out, spread, score, keys, D, bf16):
    """How far an fp32 (bf16: with weights and output rounded to bf16) result may be from `out`.

    A score is a sum of D products in fp32 (each of its D roundings, and that of the scale's product, off by
    2^-24 of at most `score`), and its exponential takes one more rounding of an argument of that size and is
    good to 2^-22: a weight is off by e = 2^-24 (D + 4) score + 2^-21 of itself (score in units of the
    exponent).  Sums of weights, and of weights times values, over `keys` terms: 2^-24 (keys + 8) each, the
    scaling of partial sums included.  So out is off by twice (numerator and denominator) e + that sum's
    error, of `spread`.  bf16: each weight's rounding of 2^-8 of itself, on the numerator, and out's own."""
    with np.errstate(invalid="ignore"):
        e = 2.0 ** -24 * (D + 4) * score + 2.0 ** -21 + 2.0 ** -24 * (keys + 8)
        bound = 2 * e * spread * 1.01 + 2.0 ** -24 * np.abs(out) + 1e-37
        if bf16:
            bound = bound + 2.0 ** -8 * spread * 1.01 + 2.0 ** -8 * np.abs(out) * 1.01
    return bound


def sample(x, u, temperature, k, p, m):
    """(token, margin): one row, in long double; margin is how far the nearest border of the draw or of a
    cut by weight is from its uniform or share, in weights of the row's largest, which is 1."""
    x = np.asarray(x, dtype=np.longdouble)
    V = len(x)
    u, temperature, p, m = (np.longdouble(np.float32(v)) for v in (u, temperature, p, m))
    if np.isnan(x).any() or not np.isfinite(x.max()) or not (0 <= u < 1) or not (0 <= temperature < np.inf) \
            or np.isnan(p) or np.isnan(m):
        return -1, 1.0
    if temperature == 0:
        return int(np.argmax(x)), 1.0
    w = np.exp((x - x.max()) / temperature)
    order = np.argsort(-x, kind="stable")
    nk = k if 1 <= k < V else V
    mass = np.cumsum(w[order])
    margin, n = np.longdouble(1), nk
    if p < 1:
        share = max(p, np.longdouble(0)) * mass[nk - 1]
        n = min(nk, int(np.searchsorted(mass[:nk], share, side="left")) + 1)
        margin = min(margin, np.abs(mass[:nk] - share).min())
    if m > 0:
        n = min(n, int((w[order] >= min(m, np.longdouble(1))).sum()))
    kept = np.zeros(V, dtype=bool)
    kept[order[:max(n, 1)]] = True
    mass = np.cumsum(np.where(kept, w, 0))
    at = u * mass[-1]
    inside = np.abs(mass - at)[np.where(kept, w, 0) > 0]
    inside = inside[:-1] if len(inside) > 1 else np.ones(1)  # the last border is the total: u < 1
    return int(np.searchsorted(mass, at, side="right")), float(min(margin, inside.min()))


def walk(tokens, parents, sampled):
    """(path, emitted) of one tree: the nodes from the root on, and the tokens drawn there; empty if faulty."""
    path, emitted, cur = [], [], 0
    if parents[0] != -1:
        return [], []
    while True:
        if sampled[cur] < 0:
            return [], []
        path.append(cur)
        emitted.append(int(sampled[cur]))
        nxt = [c for c in range(cur + 1, len(tokens)) if parents[c] == cur and tokens[c] == sampled[cur]]
        if not nxt:
            return path, emitted
        cur = nxt[0]
