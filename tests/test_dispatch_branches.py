"""Branches of the 8-bit operators and the log-probabilities that only sizes
past the other tests' reach: several units per thread in each type and
alignment, staging past the memory-side cache, rows of more than 64 parts, and
joins of many long rows."""
import numpy as np
import pytest
import torch

from tests import quant_ref as R
from tests.test_quantized_rows_and_cache import check_commit, check_read, check_rows, sv
from tests.test_token_logprobs import BF, DEV, F32, INF, NAN, compare

pytestmark = pytest.mark.gpu
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [1024, 1023])
def test_rows_by_four(d, dtype):
    """From 65536 blocks on a thread takes four units; the last block of threads is short."""
    g = torch.Generator().manual_seed(d)
    check_rows((torch.randn(8203, d, generator=g) * torch.exp(torch.randn(8203, 1, generator=g))).to(dtype).to(DEV))


@pytest.mark.parametrize("E,dtype", [(257, BF), (256, F32), (264, F32)])
def test_commits_by_four(E, dtype):
    g = torch.Generator().manual_seed(E)
    B, K, L = 40, 5, 9
    check_commit(40, B, K, L, E, dtype, torch.randint(0, K + 1, (B,), generator=g).numpy(),
                 torch.randint(0, L - K + 1, (B,), generator=g).numpy())


@pytest.mark.parametrize("E", [128, 129, 136])
def test_reads_by_four(E):
    g = torch.Generator().manual_seed(E)
    L = 75
    check_read(8, 64, L, L, E, BF, torch.randint(0, L + 1, (64,), generator=g).numpy())


@pytest.mark.parametrize("K,E,dtype", [(4100, 1024, BF), (2060, 1023, F32)])
def test_commit_of_more_than_the_memory_side_cache(K, E, dtype):
    """Staging of more than 256 MiB."""
    P, B, L = 4, 8, K + 37
    g = torch.Generator(device=DEV).manual_seed(K)
    nb = -(-E // 128)
    staging = torch.randn(P, B, K, E, generator=g, device=DEV).to(dtype)
    assert staging.numel() * staging.element_size() > 256 << 20
    codes = torch.full((P, B, L, E), 0x55, dtype=torch.uint8, device=DEV)
    scales = torch.full((P, B, L, nb), 0x55, dtype=torch.uint8, device=DEV)
    acc = torch.tensor([K, 0, 1, K - 1, K // 2, 777, K, 5], dtype=torch.int32, device=DEV)
    ln = torch.tensor([37, 3, 0, 12, 1, 36, 0, L - 5], dtype=torch.int32, device=DEV)
    st = sv().spec_kv_commit_quantized(codes.view(F8), scales.view(E8), staging, acc, ln.clone())
    assert st.tolist() == [0] * B
    want_c, want_s = sv().spec_quantize_rows(staging)     # compared with the 64-bit form by the tests of rows
    want_c, want_s = want_c.view(torch.uint8)[..., :E], want_s.view(torch.uint8)
    for b, (n, at) in enumerate(zip(acc.tolist(), ln.tolist())):
        assert torch.equal(codes[:, b, at:at + n], want_c[:, b, :n])
        assert torch.equal(scales[:, b, at:at + n], want_s[:, b, :n])
        for t in (codes, scales):
            assert (t[:, b, :at] == 0x55).all() and (t[:, b, at + n:] == 0x55).all()
    rc, rs = R.quantize(R.as_f64(staging[:, 0, K - 3:]))
    assert np.array_equal(codes[:, 0, 37 + K - 3:].cpu().numpy(), rc[..., :E])
    assert np.array_equal(scales[:, 0, 37 + K - 3:].cpu().numpy(), rs)


@pytest.mark.parametrize("dtype,V", [(BF, 1200003), (F32, 600011), (BF, 1 << 20), (BF, (1 << 20) + 1),
                                     (F32, (1 << 19) + 1)])
def test_rows_of_more_than_64_parts(dtype, V):
    """Parts of 16384 bf16 or 8192 fp32 logits, joined 64 at a time: whole groups of them masked, a fault in one."""
    group = 64 * (16384 if dtype == BF else 8192)
    g = torch.Generator().manual_seed(V)
    x = (torch.randn(8, V, generator=g) * 3).to(dtype)
    x[1, :min(group, V - 1)] = -INF                # the first 64 parts
    x[2, group - 5:] = -INF                        # what follows them, and the row's last part
    x[3, V - 1] = 90.0                             # all of the probability at the end
    x[4, 5] = 90.0
    x[5, V - 2] = NAN
    x[6, 77] = INF
    x[7] = 1.5                                     # ties
    compare_with(x, [V - 2, V - 1, 9, 4, V - 1, 3, 3, V - 1], 20)
    compare_with(x, [V - 1, V - 1, 0, V - 1, 5, V - 2, 77, 0], 0, 0.7)


def compare_with(x, tokens, top, T=1.0):
    T = float(np.float32(T))
    t = torch.tensor(tokens, dtype=torch.int32)
    got = [v.cpu().numpy() for v in sv().spec_token_logprobs(x.to(DEV), t.to(DEV), top, T)]
    compare(x, t, top, T, got)


@pytest.mark.parametrize("N,V,dtype", [(769, 66001, BF), (800, 131072, BF), (800, 33003, F32), (768, 66001, BF)])
def test_joins_of_many_long_rows(N, V, dtype):
    """Blocks of four waves join the rows from 769 on."""
    g = torch.Generator().manual_seed(N + V)
    x = (torch.randn(13, V, generator=g) * 3).to(dtype)
    x[3, :V // 2] = -INF
    x[5] = 0.25
    x[7, 40000 % V] = NAN
    x[9] = -INF
    x = x.repeat(N // 13 + 1, 1)[:N].contiguous()
    t = torch.randint(0, V, (N,), generator=g).to(torch.int32)
    t[::11] = -1
    got = [v.cpu().numpy() for v in sv().spec_token_logprobs(x.to(DEV), t.to(DEV), 20)]
    some = list(range(0, 14)) + list(range(N - 14, N))
    compare(x[some], t[some], 20, 1.0, [v[some] for v in got])
    nothing = (t < 0).numpy() | np.isin(np.arange(N) % 13, (7, 9))
    assert np.array_equal(np.isnan(got[0]), nothing)
    assert (got[2][(np.arange(N) % 13 == 5) & ~nothing] == np.arange(20)).all()
