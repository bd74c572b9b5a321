"""Rows and KV caches in the 8-bit block format against 64-bit plain forms.

Codes and scales are fully determined (x * 2^-e is exact, one rounding), and
values read back have four significant bits, so every comparison of a code, a
scale or a value is an equality."""
import numpy as np
import pytest
import torch

from tests import quant_ref as R

DEV = torch.device("cuda", 0)
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
BF, F32 = torch.bfloat16, torch.float32


def sv():
    import speculative_sampling_verification_vocab_amd as m
    return m


def special_rows(dtype):
    """Blocks where the format can go wrong: zeros, subnormals, the borders of a scale, ties, extremes, NaN."""
    g = torch.Generator().manual_seed(5)
    rows = torch.randn(16, 256, generator=g)
    rows[0] = 0.0
    rows[1] = -0.0
    rows[2, 0], rows[2, 1:] = 448.0, 1.0                      # the largest value of a scale
    rows[3, 0], rows[3, 1:] = 450.0, 1.0                      # just above (450 is a bf16 value)
    rows[4] = torch.arange(256) / 256.0 * 448.0               # every binade, ties among them
    rows[5] = torch.tensor([1.0625, 1.1875] * 128)            # ties between neighbouring codes
    rows[5, 0] = 448.0
    rows[6] = torch.finfo(dtype).max * torch.sign(rows[6])
    rows[7] = 1e-38 * rows[7]
    rows[8] = torch.finfo(torch.float32).tiny / 4 * torch.sign(rows[8])  # subnormal
    rows[9, 3] = float("nan")
    rows[10, 200], rows[10, 5] = float("inf"), float("-inf")
    rows[11, :128] = float("inf")                             # a block with nothing finite
    rows[12, 1:] = rows[12, 1:] * 1e-6                        # one value that dwarfs the rest
    rows[12, 0] = 1e6
    rows[13] = torch.finfo(dtype).min                         # the lowest value, as masks use it
    rows[14] = 2.0 ** -10 * 448.0                             # below the least code of a wide block ..
    rows[14, 7] = 448.0 * 1024
    rows[15] = -rows[4]
    return rows.to(dtype)


def check_rows(x):
    codes, scales = sv().spec_quantize_rows(x)
    torch.cuda.synchronize()
    rc, rs = R.quantize(R.as_f64(x))
    assert codes.dtype == F8 and scales.dtype == E8
    assert np.array_equal(R.as_bytes(scales), rs)
    assert R.same_codes(R.as_bytes(codes), rc)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,d", [(1, 1), (1, 128), (3, 7), (5, 127), (4, 129), (2, 136), (17, 2880), (9, 1000),
                                    (33, 4096), (1, 8192), (257, 130), (16400, 256)])
def test_rows(rows, d, dtype):
    g = torch.Generator().manual_seed(rows * 10007 + d)
    x = torch.randn(rows, d, generator=g) * torch.exp(3 * torch.randn(rows, 1, generator=g))
    print(f"case rows={rows} d={d} {dtype}", flush=True)
    check_rows(x.to(dtype).to(DEV))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_special_values(dtype):
    check_rows(special_rows(dtype).to(DEV))
    check_rows(special_rows(dtype)[:, :255].contiguous().to(DEV))   # element loads


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_off_their_alignment(dtype):
    """A base that is only element-aligned, with row lengths that would allow vectors."""
    flat = torch.randn(1 + 6 * 256, generator=torch.Generator().manual_seed(3)).to(dtype).to(DEV)
    check_rows(flat[1:].view(6, 256))


@pytest.mark.gpu
def test_every_bf16_value():
    """All 65536 bit patterns, one block each: alone in its block, and beside the value 1."""
    x = torch.zeros(2, 65536, 128, dtype=BF)
    x[:, :, 3] = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF)
    x[1, :, 9] = 1.0
    x = x.to(DEV)
    check_rows(x)


@pytest.mark.gpu
def test_rows_leave_the_rest_alone():
    x = torch.randn(7, 200, generator=torch.Generator().manual_seed(4)).to(BF).to(DEV)
    cb = torch.full((9, 256), 0x55, dtype=torch.uint8, device=DEV)
    sb = torch.full((9, 2), 0x55, dtype=torch.uint8, device=DEV)
    codes, scales = cb[1:8].view(F8), sb[1:8].view(E8)
    got = sv().spec_quantize_rows(x, out=(codes, scales))
    assert got[0] is codes and got[1] is scales
    rc, rs = R.quantize(R.as_f64(x))
    assert np.array_equal(R.as_bytes(codes), rc) and np.array_equal(R.as_bytes(scales), rs)
    for t in (cb, sb):
        assert (t[0] == 0x55).all() and (t[8] == 0x55).all()


@pytest.mark.gpu
def test_rows_of_nothing():
    codes, scales = sv().spec_quantize_rows(torch.empty(0, 64, dtype=BF, device=DEV))
    assert codes.shape == (0, 128) and scales.shape == (0, 1)


# ---- the cache ------------------------------------------------------------------

def commit_reference(codes, scales, staging, acc, ln):
    codes, scales, ln = codes.copy(), scales.copy(), ln.copy()
    status = np.zeros(len(ln), dtype=np.int32)
    P, B, K, E = staging.shape
    for b in range(B):
        n = int(acc[b])
        if not 0 <= n <= K:
            status[b] = 2
        elif ln[b] < 0 or int(ln[b]) + n > codes.shape[2]:
            status[b] = 1
        else:
            if n and E and P:
                c, s = R.quantize(staging[:, b, :n])
                codes[:, b, ln[b]:ln[b] + n] = c[..., :E]
                scales[:, b, ln[b]:ln[b] + n] = s
            ln[b] += n
    return codes, scales, ln, status


def cache(P, B, L, E, seed):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (P, B, L, E), generator=g, dtype=torch.uint8)
    scales = torch.randint(1, 255, (P, B, L, -(-E // 128)), generator=g, dtype=torch.uint8)
    return codes, scales


def check_commit(P, B, K, L, E, dtype, acc, ln, seed=1, apart=True, shift=0):
    codes, scales = cache(P, B, L, E, seed)
    g = torch.Generator().manual_seed(seed + 1)
    staging = torch.randn(P, B, K, E, generator=g).to(dtype)
    acc, ln = np.asarray(acc, dtype=np.int32), np.asarray(ln, dtype=np.int32)
    want = commit_reference(codes.numpy(), scales.numpy(), R.as_f64(staging), acc, ln)
    st = staging.to(DEV)
    if shift:  # a staging buffer that begins `shift` elements into its allocation
        buf = torch.empty(staging.numel() + shift, dtype=dtype, device=DEV)
        buf[shift:] = st.flatten()
        st = buf[shift:].view(staging.shape)
    c, s = codes.to(DEV), scales.to(DEV)
    a, l = torch.from_numpy(acc).to(DEV), torch.from_numpy(ln).to(DEV)
    new = torch.full((B,), -77, dtype=torch.int32, device=DEV) if apart else None
    status = sv().spec_kv_commit_quantized(c.view(F8), s.view(E8), st, a, l, new_len=new)
    torch.cuda.synchronize()
    assert np.array_equal(status.cpu().numpy(), want[3])
    assert np.array_equal((new if apart else l).cpu().numpy(), want[2])
    if apart:
        assert np.array_equal(l.cpu().numpy(), ln)
    assert np.array_equal(s.cpu().numpy(), want[1])
    assert np.array_equal(c.cpu().numpy(), want[0])  # finite staging: no NaN code is written


@pytest.mark.gpu
@pytest.mark.parametrize("apart", [True, False])
@pytest.mark.parametrize("P,B,K,L,E,dtype", [
    (4, 16, 7, 40, 64, BF),        # rows shorter than a block
    (6, 8, 5, 24, 1024, BF),
    (3, 12, 4, 20, 33, BF),        # odd rows: element accesses
    (2, 9, 6, 30, 576, F32),       # a last block of 64
    (5, 7, 3, 16, 12, F32),        # rows of 12: element accesses
    (1, 300, 2, 8, 8, BF),         # more sequences than a block of threads
    (2, 3, 300, 700, 136, BF),     # a prompt's length
    (64, 40, 7, 12, 1024, BF),     # several units per thread
    (40, 40, 5, 9, 257, F32),      # the same, odd rows
])
def test_commits(P, B, K, L, E, dtype, apart):
    print(f"case P={P} B={B} K={K} L={L} E={E} {dtype} apart={apart}", flush=True)
    g = torch.Generator().manual_seed(P * 1000 + B * 10 + K)
    acc = torch.randint(-1, K + 2, (B,), generator=g).numpy()
    ln = torch.randint(-1, L + 2, (B,), generator=g).numpy()
    check_commit(P, B, K, L, E, dtype, acc, ln, apart=apart)


@pytest.mark.gpu
def test_commit_one_token_and_full_caches():
    check_commit(2, 1, 1, 1, 128, BF, [1], [0])
    check_commit(2, 1, 1, 1, 128, BF, [1], [1])
    check_commit(2, 4, 3, 5, 128, BF, [3, 3, 0, 2147483647], [2, 3, 5, 1])
    check_commit(2, 3, 3, 5, 128, BF, [1, 2, 3], [2147483647, -2147483648, 5])


@pytest.mark.gpu
def test_commit_off_alignment():
    check_commit(3, 5, 4, 9, 256, BF, [4, 3, 2, 1, 0], [0, 1, 2, 3, 4], shift=1)
    check_commit(3, 5, 4, 9, 256, F32, [4, 3, 2, 1, 0], [0, 1, 2, 3, 4], shift=3)


@pytest.mark.gpu
@pytest.mark.parametrize("apart", [True, False])
def test_commit_without_planes_or_drafts(apart):
    check_commit(0, 4, 3, 10, 8, BF, [0, 1, 3, 4], [2, 9, 5, 0], apart=apart)
    check_commit(2, 3, 0, 10, 8, BF, [0, 0, 1], [3, 10, 4], apart=apart)
    check_commit(2, 3, 2, 10, 0, BF, [0, 2, 1], [3, 9, 4], apart=apart)


@pytest.mark.gpu
def test_commit_special_values():
    x = special_rows(BF).view(1, 16, 1, 256)
    codes, scales = cache(1, 16, 3, 256, 8)
    c, s = codes.to(DEV), scales.to(DEV)
    one = torch.ones(16, dtype=torch.int32, device=DEV)
    sv().spec_kv_commit_quantized(c.view(F8), s.view(E8), x.to(DEV), one, one.clone())
    rc, rs = R.quantize(R.as_f64(x))
    assert np.array_equal(s[:, :, 1:2].cpu().numpy(), rs)
    assert R.same_codes(c[:, :, 1:2].cpu().numpy(), rc)


def check_read(P, B, L, Lo, E, dtype, ln, seed=2, shift=0):
    codes, scales = cache(P, B, L, E, seed)
    ln = np.asarray(ln, dtype=np.int32)
    mark = 7.0
    n = P * B * Lo * E
    buf = torch.full((n + shift,), mark, dtype=dtype, device=DEV)
    out = buf[shift:].view(P, B, Lo, E)
    c, s = codes.to(DEV), scales.to(DEV)
    status = sv().spec_kv_read_quantized(c.view(F8), s.view(E8), torch.from_numpy(ln).to(DEV), out)
    torch.cuda.synchronize()
    bad = (ln < 0) | (ln > min(L, Lo))
    assert np.array_equal(status.cpu().numpy(), bad.astype(np.int32))
    want = torch.full((P, B, Lo, E), mark, dtype=dtype)
    # fp32 holds every value (four bits at 2^-135 and above: subnormals too); rounding it to bf16 is torch's
    v = torch.from_numpy(R.values(codes.numpy(), scales.numpy())).float().to(dtype)
    for b in range(B):
        if not bad[b]:
            want[:, b, :ln[b]] = v[:, b, :ln[b]]
    got = out.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got, nan=0.0), torch.nan_to_num(want, nan=0.0))
    assert (buf[:shift] == mark).all()


@pytest.mark.gpu
@pytest.mark.parametrize("P,B,L,Lo,E,dtype", [
    (2, 5, 40, 40, 64, BF), (2, 3, 33, 50, 1024, BF), (2, 4, 21, 9, 33, BF), (1, 6, 17, 17, 576, F32),
    (3, 2, 11, 30, 12, F32), (1, 300, 4, 4, 8, BF), (4, 40, 300, 260, 128, BF), (4, 40, 30, 26, 1030, F32)])
def test_reads(P, B, L, Lo, E, dtype):
    print(f"case P={P} B={B} L={L} Lo={Lo} E={E} {dtype}", flush=True)
    g = torch.Generator().manual_seed(P + B * 10 + L)
    check_read(P, B, L, Lo, E, dtype, torch.randint(-1, L + 2, (B,), generator=g).numpy())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_read_every_code_and_scale(dtype):
    """Every code with every scale byte the commit writes (1 .. 248) and the rest of e8m0's finite ones."""
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).repeat(1, 1, 255, 1)   # [1, 1, 255, 256]
    scales = torch.arange(255, dtype=torch.int32).to(torch.uint8).view(1, 1, 255, 1).repeat(1, 1, 1, 2)
    out = torch.empty(1, 1, 255, 256, dtype=dtype, device=DEV)
    ln = torch.full((1,), 255, dtype=torch.int32, device=DEV)
    sv().spec_kv_read_quantized(codes.to(DEV).view(F8), scales.contiguous().to(DEV).view(E8), ln, out)
    want = torch.from_numpy(R.values(codes.numpy(), scales.numpy())).float().to(dtype)
    got = out.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got, nan=0.0), torch.nan_to_num(want, nan=0.0))


@pytest.mark.gpu
def test_read_edges():
    check_read(2, 4, 5, 5, 128, BF, [0, 1, 5, 6])
    check_read(2, 3, 5, 3, 128, F32, [3, 4, -1])
    check_read(2, 3, 5, 5, 128, BF, [5, 3, 1], shift=1)
    check_read(2, 3, 5, 5, 64, F32, [5, 3, 1], shift=2)
    check_read(0, 3, 5, 5, 64, F32, [5, 6, 1])
    check_read(2, 3, 0, 5, 64, F32, [0, 1, 0])
    check_read(2, 3, 5, 5, 0, F32, [5, 6, 1])


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    """A cache of more than 2^32 codes: its last entries are committed and read back."""
    P, B, L, E = 1, 2, (1 << 21) + 5, 1032
    codes = torch.empty(P, B, L, E, dtype=torch.uint8, device=DEV)
    scales = torch.empty(P, B, L, 9, dtype=torch.uint8, device=DEV)
    K = 3
    x = torch.randn(P, B, K, E, generator=torch.Generator().manual_seed(6)).to(BF)
    acc = torch.tensor([2, 3], dtype=torch.int32, device=DEV)
    ln = torch.tensor([L - 2, L - 3], dtype=torch.int32, device=DEV)
    assert sv().spec_kv_commit_quantized(codes.view(F8), scales.view(E8), x.to(DEV), acc, ln).tolist() == [0, 0]
    assert ln.tolist() == [L, L]
    rc, rs = R.quantize(R.as_f64(x))
    for b, n in ((0, 2), (1, 3)):
        assert np.array_equal(codes[0, b, L - n:].cpu().numpy(), rc[0, b, :n, :E])
        assert np.array_equal(scales[0, b, L - n:].cpu().numpy(), rs[0, b, :n])
    # read with the first sequence empty, so that only the far one is written
    out = torch.empty(P, B, L, E, dtype=BF, device=DEV)
    far = torch.tensor([0, L], dtype=torch.int32, device=DEV)
    assert sv().spec_kv_read_quantized(codes.view(F8), scales.view(E8), far, out).tolist() == [0, 0]
    got = R.as_f64(out[0, 1, L - 3:])
    assert np.array_equal(got, R.values(rc[0, 1, :, :E], rs[0, 1]))


# ---- refusals (no GPU) ------------------------------------------------------------

def lib():
    from speculative_sampling_verification_vocab_amd import _native
    return _native.load()


OK, INVALID, UNSUP, WS = 0, 1, 2, 3


def test_rows_refusals():
    import ctypes
    f, p = lib().spec_quantize_rows, ctypes.c_void_p

    def call(x=0x10000, R=4, d=64, dt=1, codes=0x20000, scales=0x30001):
        return f(p(x), R, d, dt, p(codes), p(scales), None)
    assert call(x=None) == INVALID and call(codes=None) == INVALID and call(scales=None) == INVALID
    assert call(R=-1) == INVALID and call(d=0) == INVALID and call(d=-3) == INVALID and call(dt=2) == INVALID
    assert call(x=0x10001) == INVALID and call(codes=0x20008) == INVALID
    assert call(x=0x10002, dt=0) == INVALID
    assert call(R=0, x=None, codes=None, scales=None) == OK
    assert call(R=0x7fffffff, d=1) == UNSUP
    assert call(R=1 << 20, d=0x7fffffff) == UNSUP


def test_commit_refusals():
    import ctypes
    f, p = lib().spec_kv_commit_quantized, ctypes.c_void_p
    ok = dict(codes=0x100000, scales=0x200001, staging=0x300000, acc=0x400000, ln=0x500000, new=0x600000,
              status=None, P=4, B=2, K=3, L=16, E=64, dt=1)

    def call(**o):
        a = {**ok, **o}
        return f(p(a["codes"]), p(a["scales"]), p(a["staging"]), p(a["acc"]), p(a["ln"]), p(a["new"]), p(a["status"]),
                 a["P"], a["B"], a["K"], a["L"], a["E"], a["dt"], None)
    for name in ("codes", "scales", "staging", "acc", "ln", "new"):
        assert call(**{name: None}) == INVALID, name
    for name in ("P", "B", "K", "L", "E"):
        assert call(**{name: -1}) == INVALID, name
    assert call(dt=7) == INVALID
    assert call(staging=0x300001) == INVALID and call(staging=0x300002, dt=0) == INVALID
    for name in ("acc", "ln", "new", "status"):
        assert call(**{name: 0x700002}) == INVALID, name
    # lengths that some blocks write while others read them
    assert call(new=0x500004) == INVALID                  # overlaps cache_len without being it
    assert call(new=0x400000) == INVALID                  # is accepted_len
    assert call(status=0x600004) == INVALID and call(status=0x500000) == INVALID and call(status=0x400004) == INVALID
    assert call(new=0x500000, status=0x500004) == INVALID
    assert call(B=0, codes=None, acc=None) == OK
    assert call(P=0x7fffffff) == UNSUP                    # more (plane, sequence) pairs than blocks
    assert call(K=0x7fffffff, L=0x7fffffff, E=1 << 20) == UNSUP
    assert call(L=0x7fffffff, E=0x7fffffff, P=1 << 10, B=1 << 10) == INVALID   # byte counts overflow


def test_read_refusals():
    import ctypes
    f, p = lib().spec_kv_read_quantized, ctypes.c_void_p
    ok = dict(codes=0x100000, scales=0x200001, ln=0x500000, out=0x600000, status=None, P=4, B=2, L=16, Lo=16, E=64,
              dt=1)

    def call(**o):
        a = {**ok, **o}
        return f(p(a["codes"]), p(a["scales"]), p(a["ln"]), p(a["out"]), p(a["status"]), a["P"], a["B"], a["L"],
                 a["Lo"], a["E"], a["dt"], None)
    for name in ("codes", "scales", "ln", "out"):
        assert call(**{name: None}) == INVALID, name
    for name in ("P", "B", "L", "Lo", "E"):
        assert call(**{name: -1}) == INVALID, name
    assert call(dt=2) == INVALID and call(out=0x600001) == INVALID and call(ln=0x500002) == INVALID
    assert call(status=0x500004) == INVALID               # overlaps cache_len
    assert call(B=0, codes=None, ln=None) == OK
    assert call(P=0x7fffffff, B=0x7fffffff) == UNSUP
    assert call(L=0x7fffffff, Lo=0x7fffffff, E=1 << 20) == UNSUP


def test_cpu_tensors_are_refused():
    m = sv()
    c, s = torch.zeros(1, 2, 4, 64, dtype=torch.uint8).view(F8), torch.zeros(1, 2, 4, 1, dtype=torch.uint8).view(E8)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        m.spec_quantize_rows(torch.zeros(2, 64, dtype=BF))
    with pytest.raises(ValueError):
        m.spec_kv_commit_quantized(c, s, torch.zeros(1, 2, 3, 64, dtype=BF), i, i)
    with pytest.raises(ValueError):
        m.spec_kv_read_quantized(c, s, i, torch.zeros(1, 2, 4, 64, dtype=BF))


@pytest.mark.gpu
def test_shapes_and_types_are_checked():
    m = sv()
    x = torch.zeros(4, 64, dtype=BF, device=DEV)
    for bad in (x.half(), x.t(), torch.zeros(4, 0, dtype=BF, device=DEV), torch.zeros((), dtype=BF, device=DEV)):
        with pytest.raises(ValueError):
            m.spec_quantize_rows(bad)
    q, e = m.spec_quantize_rows(x)
    for out in ((q,), (q[:3], e), (q, e[:3]), (q.view(torch.uint8), e)):
        with pytest.raises(ValueError):
            m.spec_quantize_rows(x, out=out)
    c = torch.zeros(1, 2, 4, 64, dtype=torch.uint8, device=DEV).view(F8)
    s = torch.zeros(1, 2, 4, 1, dtype=torch.uint8, device=DEV).view(E8)
    i = torch.zeros(2, dtype=torch.int32, device=DEV)
    st = torch.zeros(1, 2, 3, 64, dtype=BF, device=DEV)
    for args in ((c.view(torch.uint8), s, st, i, i), (c, s[:, :, :3], st, i, i), (c, s, st[..., :32], i, i),
                 (c, s, st.half(), i, i), (c, s, st, i.long(), i), (c, s, st, i, i[:1]), (c, s, st[:, :1], i, i)):
        with pytest.raises(ValueError):
            m.spec_kv_commit_quantized(*args)
    with pytest.raises(ValueError):
        m.spec_kv_commit_quantized(c, s, st, i, i, new_len=i.long())
    with pytest.raises(m.SpecVerifyError):
        m.spec_kv_commit_quantized(c, s, st, i, i)        # accepted_len and the lengths in one tensor
    out = torch.zeros(1, 2, 4, 64, dtype=BF, device=DEV)
    for args in ((c, s, i, out.half()), (c, s, i, out[..., :32]), (c, s, i[:1], out), (c, s, i, out[:, :1]),
                 (c, s, i, out.transpose(0, 1))):
        with pytest.raises(ValueError):
            m.spec_kv_read_quantized(*args)
