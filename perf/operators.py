"""Timed cases of the 8-bit and log-probability operators.

Five operators of a speculative-decoding server's step: the log-probabilities
it reports for the tokens it emits (with entropy and top alternatives), the
8-bit block format for rows, the drafter head on weights in that format, and
the KV cache committed and read back in it.

The format: e4m3 codes with one power-of-two scale for each block of 128
values along the last dimension.  A block's exponent e is the smallest integer
>= -126 with max |x| <= 448 * 2^e over its finite values; the scale is the
e8m0 byte e + 127; a code is x * 2^-e rounded to nearest even; values that are
not finite become NaN codes.

`own` False computes the plain forms (elementary torch operations in 32 bits),
`own` True calls the framework.
"""
import math

import torch

own = False

BLOCK = 128
_F = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}


# ---- the cases ------------------------------------------------------------------

def listed():
    return [
        # One sequence's verify step, 4 drafts, a 32000-token vocabulary: the smallest call, latency counts.
        {"name": "logprobs_b1_k4_v32000_f32", "op": "logprobs", "B": 1, "K": 4, "V": 32000, "dtype": "f32",
         "top": 5, "T": 1.0, "skip": True, "masked": False},
        # A small batch with sampling at T = 0.75, a grammar that masks half the vocabulary, and the widest list
        # of alternatives that serving interfaces offer.
        {"name": "logprobs_b8_k5_v128256_bf16", "op": "logprobs", "B": 8, "K": 5, "V": 128256, "dtype": "bf16",
         "top": 20, "T": 0.75, "skip": True, "masked": True},
        # The benchmark's batch: 256 sequences, 7 drafts, 262144 tokens; rows after a first rejection carry no token.
        {"name": "logprobs_b256_k7_v262144_bf16", "op": "logprobs", "B": 256, "K": 7, "V": 262144, "dtype": "bf16",
         "top": 20, "T": 1.0, "skip": True, "masked": False},
        # The hidden states of 128 draft positions, as a head quantises them on each step.
        {"name": "quantize_128x4096_bf16", "op": "quantize", "rows": 128, "d": 4096, "dtype": "bf16"},
        # A whole head weight, once at load time.
        {"name": "quantize_128256x4096_bf16", "op": "quantize", "rows": 128256, "d": 4096, "dtype": "bf16"},
        # One sequence's 5 draft positions on a narrow shortlist of 16 clusters of 501 tokens.
        {"name": "head_m5_n8016_d4096", "op": "head", "M": 5, "d": 4096, "V": 128256, "cs": 501, "n_sel": 16,
         "out": "f32"},
        # 128 positions on a frequency-ranked shortlist of 32768 scattered tokens.
        {"name": "head_m128_n32768_d4096", "op": "head", "M": 128, "d": 4096, "V": 128256, "cs": 1, "n_sel": 32768,
         "out": "bf16"},
        # A full vocabulary for 256 sequences of 7 positions: the largest product.
        {"name": "head_m1792_n128256_d4096", "op": "head", "M": 1792, "d": 4096, "V": 128256, "cs": 501,
         "n_sel": 256, "out": "bf16"},
        # One sequence's accepted drafts, 32 layers of keys and values.
        {"name": "kv_commit_b1_k5_p64_e1024", "op": "kv_commit", "P": 64, "B": 1, "K": 5, "L": 2048, "E": 1024,
         "dtype": "bf16"},
        # The benchmark's commit batch.
        {"name": "kv_commit_b256_k7_p64_e1024", "op": "kv_commit", "P": 64, "B": 256, "K": 7, "L": 64, "E": 1024,
         "dtype": "bf16"},
        # One layer's keys and values of one short sequence, read back for its attention.
        {"name": "kv_read_b1_l512_e1024", "op": "kv_read", "P": 2, "B": 1, "L": 512, "E": 1024, "dtype": "bf16"},
        # One layer's keys and values of 64 sequences of up to 8192 tokens.
        {"name": "kv_read_b64_l8192_e1024", "op": "kv_read", "P": 2, "B": 64, "L": 8192, "E": 1024,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logprobs", "quantize", "head", "kv_commit", "kv_read"])
    if op == "logprobs":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        K, V = rng.randint(0, 8), _log(rng, 8000, 262144)
        most = (1 << 30) // (_SIZE[dtype] * V * (K + 1))
        return {"op": op, "B": _log(rng, 1, min(256, most)), "K": K, "V": V, "dtype": dtype,
                "top": rng.choice([0, 1, 5, 20, rng.randint(2, 20)]), "T": rng.randint(32, 96) / 64,
                "skip": rng.random() < 0.7, "masked": rng.random() < 0.3}
    if op == "quantize":
        d = rng.choice([2048, 4096, 5120, 8192, _log(rng, 64, 8192)])
        return {"op": op, "rows": _log(rng, 1, min(262144, (1 << 29) // d)), "d": d,
                "dtype": rng.choice(["bf16", "bf16", "f32"])}
    if op == "head":
        d = rng.choice([2048, 4096, 5120, _log(rng, 256, 8192)])
        cs = rng.choice([1, 1, 501, 167, 128, rng.randint(2, 600)])
        clusters = max(1, _log(rng, 2000, min(151936, (1 << 29) // d)) // cs)
        return {"op": op, "M": _log(rng, 1, 1792), "d": d, "V": clusters * cs, "cs": cs,
                "n_sel": rng.randint(max(1, clusters // 8), clusters), "out": rng.choice(["bf16", "f32"])}
    dtype, E = rng.choice(["bf16", "bf16", "f32"]), rng.choice([128, 512, 576, 1024, 2048, _log(rng, 64, 2048)])
    if op == "kv_commit":
        P, K = 2 * rng.randint(1, 32), rng.choice([rng.randint(1, 8), _log(rng, 1, 2048)])
        B = _log(rng, 1, max(1, min(256, (1 << 27) // (P * K * E))))
        L = K + _log(rng, 16, 1024)
        while P * B * L * E > 1 << 30 and L > K + 16:
            L = max(K + 16, L // 2)
        return {"op": op, "P": P, "B": B, "K": K, "L": L, "E": E, "dtype": dtype}
    P, L = 2 * rng.randint(1, 2), _log(rng, 1, 16384)
    return {"op": op, "P": P, "B": _log(rng, 1, max(1, min(256, (1 << 29) // (P * L * E)))), "L": L, "E": E,
            "dtype": dtype}


# ---- inputs ---------------------------------------------------------------------

def _spread(case, seed, most):
    """B whole numbers that run evenly over 0..most, in an order of the seed."""
    g = torch.Generator().manual_seed(seed)
    B = case["B"]
    v = torch.arange(B) * (most + 1) // B if B > 1 else torch.tensor([most - most // 4])
    return v[torch.randperm(B, generator=g)]


def _codes(shape, g):
    """Cache contents written earlier: finite e4m3 codes, scales around 2^-8."""
    codes = torch.randint(0, 254, shape, generator=g, device="cuda", dtype=torch.uint8)
    codes += (codes >= 127).to(torch.uint8)  # 0x7f is NaN; 254 is the last code used, 0xff is NaN too
    blocks = -(-shape[-1] // BLOCK)
    scales = torch.randint(115, 123, shape[:-1] + (blocks,), generator=g, device="cuda", dtype=torch.uint8)
    return codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)
    op, s = case["op"], dict(case)
    dtype = _F[case.get("dtype", "bf16")]
    if op == "logprobs":
        B, K, V = case["B"], case["K"], case["V"]
        x = torch.randn((B, K + 1, V), generator=g, device="cuda").mul_(3.0)
        x -= torch.log(torch.arange(1, V + 1, device="cuda", dtype=torch.float32))
        if case["masked"]:
            x[torch.rand((B, 1, V), generator=g, device="cuda").expand_as(x) < 0.5] = -math.inf
        u = torch.rand((B, K + 1, V), generator=g, device="cuda").clamp_(1e-9, 1 - 1e-6)
        tokens = (x / case["T"] - torch.log(-torch.log(u))).argmax(-1).to(torch.int32)
        if case["skip"]:  # what a verify step leaves: the tokens up to the first rejection, then -1
            n = _spread(case, seed, K).to("cuda")
            tokens = torch.where(torch.arange(K + 1, device="cuda") <= n[:, None], tokens, -1).to(torch.int32)
        s["logits"], s["tokens"] = x.to(dtype), tokens.contiguous()
    elif op == "quantize":
        x = torch.randn((case["rows"], case["d"]), generator=g, device="cuda")
        s["x"] = (x * torch.exp(torch.randn((case["rows"], 1), generator=g, device="cuda"))).to(dtype)
    elif op == "head":
        clusters = case["V"] // case["cs"]
        s["h"] = torch.randn((case["M"], case["d"]), generator=g, device="cuda").to(torch.bfloat16)
        W = torch.randn((case["V"], case["d"]), generator=g, device="cuda").mul_(case["d"] ** -0.5)
        s["codes"], s["scales"] = _plain_quantize(W.to(torch.bfloat16))
        s["ids"] = torch.randperm(clusters, generator=g, device="cuda")[:case["n_sel"]].sort()[0].to(torch.int32)
    else:
        P, B, L, E = case["P"], case["B"], case["L"], case["E"]
        s["codes"], s["scales"] = _codes((P, B, L, E), g)
        if op == "kv_commit":
            K = case["K"]
            s["staging"] = torch.randn((P, B, K, E), generator=g, device="cuda").to(dtype)
            s["accepted"] = _spread(case, seed, K).to(torch.int32).cuda()
            s["len"] = torch.randint(0, L - K + 1, (B,), generator=g, device="cuda").to(torch.int32)
            s["new_len"] = torch.empty_like(s["len"])
        else:
            s["len"] = _read_lengths(case, seed).to(torch.int32).cuda()
            s["rows"] = torch.zeros((P, B, L, E), device="cuda", dtype=dtype)
    return s


def _read_lengths(case, seed):
    """Lengths from half of L to L."""
    return case["L"] - _spread(case, seed, case["L"] // 2)


# ---- the plain forms ------------------------------------------------------------

def _plain_quantize(x):
    """e4m3 codes [..., D] (D: the last dimension up to a whole block) and e8m0 scales."""
    d = x.shape[-1]
    blocks = -(-d // BLOCK)
    v = x.float()
    if blocks * BLOCK > d:
        v = torch.cat([v, v.new_zeros(v.shape[:-1] + (blocks * BLOCK - d,))], -1)
    v = v.view(v.shape[:-1] + (blocks, BLOCK))
    finite = torch.isfinite(v)
    amax = torch.where(finite, v, 0.0).abs().amax(-1, keepdim=True)
    m, k = torch.frexp(amax)  # amax = m * 2^k; 448 = 0.875 * 2^9
    e = torch.where(amax > 0, k - 9 + (m > 0.875).to(k.dtype), -126).clamp(min=-126)
    inverse = ((127 - e) << 23).to(torch.int32).view(torch.float32)
    q = (torch.where(finite, v, math.nan) * inverse).to(torch.float8_e4m3fn)
    return q.flatten(-2), (e + 127).to(torch.uint8).squeeze(-1).view(torch.float8_e8m0fnu)


def _plain_values(codes, scales):
    """The 32-bit values that codes [..., E] with scales [..., ceil(E / 128)] stand for."""
    e = scales.view(torch.uint8).to(torch.int32)
    step = (e << 23).view(torch.float32).repeat_interleave(BLOCK, -1)[..., :codes.shape[-1]]
    return codes.float() * step


def _plain_logprobs(s):
    x = s["logits"].float()
    V, top, tok = s["V"], s["top"], s["tokens"].long()
    live = (tok >= 0) & (tok < V)
    z = x / s["T"]
    peak = z.amax(-1, keepdim=True)
    z = z - peak
    e = torch.exp(z)
    total = e.sum(-1)
    lse = torch.log(total)
    logprob = z.gather(-1, tok.clamp(0, V - 1)[..., None])[..., 0] - lse
    entropy = lse - torch.where(e > 0, e * z, 0.0).sum(-1) / total
    # Alternatives by (value, lower id): one whole number per token that orders them.
    bits = (x + 0.0).view(torch.int32)
    order = (bits ^ ((bits >> 31) & 0x7fffffff)).to(torch.int64)
    order = (order << 30) + (V - 1 - torch.arange(V, device=x.device))
    best = order.topk(min(top, V), -1, largest=True, sorted=True)[1]
    found = x.gather(-1, best) > -math.inf
    top_lp = torch.where(found, z.gather(-1, best) - lse[..., None], -math.inf)
    ids = torch.where(found, best, -1)
    gone = ~live[..., None]
    return {"logprob": torch.where(live, logprob, math.nan), "entropy": torch.where(live, entropy, math.nan),
            "top_ids": torch.where(gone, -1, ids).to(torch.int32), "top_logprobs": torch.where(gone, math.nan, top_lp)}


def _plain_head(s):
    h = _plain_values(*_plain_quantize(s["h"]))
    rows = (s["ids"].long()[:, None] * s["cs"] + torch.arange(s["cs"], device="cuda")).flatten()
    W = _plain_values(s["codes"].view(torch.uint8)[rows].view(torch.float8_e4m3fn),
                      s["scales"].view(torch.uint8)[rows].view(torch.float8_e8m0fnu))
    return {"logits": (h @ W.t()).to(_F[s["out"]])}


def _plain_commit(s):
    n, at, K, L, E = s["accepted"].long(), s["len"].long(), s["K"], s["L"], s["E"]
    status = torch.where((n < 0) | (n > K), 2, torch.where((at < 0) | (at + n > L), 1, 0))
    takes = (status == 0)[:, None] & (torch.arange(K, device=n.device) < n[:, None])
    b, j = takes.nonzero(as_tuple=True)
    q, e = _plain_quantize(s["staging"][:, b, j])
    s["codes"].view(torch.uint8)[:, b, at[b] + j] = q.view(torch.uint8)[..., :E]
    s["scales"].view(torch.uint8)[:, b, at[b] + j] = e.view(torch.uint8)
    s["new_len"].copy_(torch.where(status == 0, at + n, at))
    return {"codes": s["codes"], "scales": s["scales"], "len": s["new_len"], "status": status.to(torch.int32)}


def _plain_read(s):
    n, L = s["len"].long(), s["L"]
    status = ((n < 0) | (n > L)).to(torch.int32)
    there = (status == 0)[:, None] & (torch.arange(L, device=n.device) < n[:, None])
    values = _plain_values(s["codes"], s["scales"]).to(s["rows"].dtype)
    s["rows"].copy_(torch.where(there[None, :, :, None], values, s["rows"]))
    return {"rows": s["rows"], "status": status}


# ---- one pass -------------------------------------------------------------------

def run(s):
    op = s["op"]
    if not own:
        if op == "quantize":
            codes, scales = _plain_quantize(s["x"])
            return {"codes": codes, "scales": scales}
        return {"logprobs": _plain_logprobs, "head": _plain_head, "kv_commit": _plain_commit,
                "kv_read": _plain_read}[op](s)
    import speculative_sampling_verification_vocab_amd as sv
    if op == "logprobs":
        got = sv.spec_token_logprobs(s["logits"], s["tokens"], s["top"], s["T"])
        return dict(zip(("logprob", "entropy", "top_ids", "top_logprobs"), got))
    if op == "quantize":
        codes, scales = sv.spec_quantize_rows(s["x"])
        return {"codes": codes, "scales": scales}
    if op == "head":
        return {"logits": sv.spec_draft_head_quantized(s["h"], s["codes"], s["scales"], s["ids"], s["cs"],
                                                       dtype=_F[s["out"]])}
    if op == "kv_commit":
        status = sv.spec_kv_commit_quantized(s["codes"], s["scales"], s["staging"], s["accepted"], s["len"],
                                             new_len=s["new_len"])
        return {"codes": s["codes"], "scales": s["scales"], "len": s["new_len"], "status": status}
    status = sv.spec_kv_read_quantized(s["codes"], s["scales"], s["len"], s["rows"])
    return {"rows": s["rows"], "status": status}


# ---- what a pass cannot do without ----------------------------------------------

def work(case):
    op, size = case["op"], _SIZE[case.get("dtype", "bf16")]
    if op == "logprobs":
        rows = case["B"] * (case["K"] + 1)
        live = int((_spread(case, 0, case["K"]) + 1).sum()) if case["skip"] else rows
        # per element: scale, subtract, exponential, two sums and a product; comparisons are not counted
        return {"bytes": live * case["V"] * size + rows * (12 + 8 * case["top"]), "flops": 6 * live * case["V"]}
    if op == "quantize":
        blocks = -(-case["d"] // BLOCK)
        return {"bytes": case["rows"] * (case["d"] * size + blocks * (BLOCK + 1)),
                "flops": 2 * case["rows"] * case["d"]}
    if op == "head":
        N, blocks = case["n_sel"] * case["cs"], -(-case["d"] // BLOCK)
        return {"bytes": N * (case["d"] + blocks) + case["M"] * case["d"] * 2 + 4 * case["n_sel"] +
                case["M"] * N * _SIZE[case["out"]], "flops": 2 * case["M"] * N * case["d"]}
    E, blocks = case["E"], -(-case["E"] // BLOCK)
    if op == "kv_commit":
        entries = case["P"] * int(_spread(case, 0, case["K"]).sum())
        return {"bytes": entries * (E * size + E + blocks) + 16 * case["B"], "flops": 2 * entries * E}
    entries = case["P"] * int(_read_lengths(case, 0).sum())
    return {"bytes": entries * (E * size + E + blocks) + 8 * case["B"], "flops": entries * E}


# ---- the definitions in 64 bits -------------------------------------------------

def _exact_quantize(x):
    """(values of the codes, scales) in 64 bits, from the definition: the block's
    exponent by comparison with 448 * 2^e, the code by rounding to its own step."""
    d = x.shape[-1]
    v = torch.nn.functional.pad(x.double(), (0, -d % BLOCK)).unflatten(-1, (-1, BLOCK))
    biggest = torch.nan_to_num(v, nan=0.0, posinf=0.0, neginf=0.0).abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(biggest.clamp(min=2.0 ** -140) / 448.0))
    e = torch.where(biggest > 448.0 * torch.exp2(e), e + 1, e)
    e = torch.where(biggest <= 448.0 * torch.exp2(e - 1), e - 1, e).clamp(min=-126.0)
    v = torch.where(v.isfinite(), v, math.nan) / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))).clamp(min=-6.0) - 3.0)
    return (torch.round(v / step) * step).flatten(-2), torch.exp2(e)[..., 0]


def _exact_values(codes, scales):
    step = scales.double()[..., None].expand(scales.shape + (BLOCK,)).flatten(-2)
    return codes.double() * step[..., :codes.shape[-1]]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        codes, scales = _exact_quantize(s["x"])
        return {"codes": codes, "scales": scales}
    if op == "logprobs":
        x, tok = s["logits"].double(), s["tokens"].long()
        dead = (tok < 0) | (tok >= case["V"])
        lp = x / case["T"]
        lp = lp - torch.logsumexp(lp, -1, keepdim=True)
        entropy = -(lp.exp() * lp.clamp(min=-1e6)).sum(-1)
        values, ids = torch.sort(x, dim=-1, descending=True, stable=True)
        ids = ids[..., :case["top"]].clone()
        ids[values[..., :case["top"]] == -math.inf] = -1
        del values
        top = torch.where(ids >= 0, lp.gather(-1, ids.clamp(min=0)), -math.inf)
        chosen = lp.gather(-1, tok.clamp(min=0)[..., None])[..., 0]
        chosen[dead], entropy[dead], ids[dead], top[dead] = math.nan, math.nan, -1, math.nan
        return {"logprob": chosen, "entropy": entropy, "top_ids": ids, "top_logprobs": top}
    if op == "head":
        codes, scales = _exact_quantize(s["h"])
        h = _exact_values(codes, scales)
        keep = torch.zeros(case["V"] // case["cs"], dtype=torch.bool, device="cuda")
        keep[s["ids"].long()] = True
        keep = keep.repeat_interleave(case["cs"]).nonzero()[:, 0]
        W = _exact_values(s["codes"].float()[keep], s["scales"].float()[keep])
        return {"logits": torch.matmul(h, W.t().contiguous())}
    if op == "kv_commit":
        values, steps = _exact_quantize(s["staging"])
        codes, scales, new_len = s["codes"].double(), s["scales"].double(), s["len"].clone()
        for b, (n, at) in enumerate(zip(s["accepted"].tolist(), s["len"].tolist())):
            codes[:, b, at:at + n] = values[:, b, :n, :case["E"]]
            scales[:, b, at:at + n] = steps[:, b, :n]
            new_len[b] = at + n
        return {"codes": codes, "scales": scales, "len": new_len,
                "status": torch.zeros_like(new_len)}
    rows = _exact_values(s["codes"], s["scales"])
    for b, n in enumerate(s["len"].tolist()):
        rows[:, b, n:] = 0.0
    return {"rows": rows, "status": torch.zeros_like(s["len"])}
