"""A cache of no rows (its tensors are empty): the commits set status and
lengths, as for any other cache that has no room."""
import ctypes

import pytest
import torch

import speculative_sampling_verification_vocab_amd as sv

DEV = torch.device("cuda", 0)


def test_a_cache_without_rows_needs_no_buffer():
    """Checked on the host: the null buffers are accepted, so the calls get as far as their launch (which fails
    where there is no GPU) or are refused for another argument."""
    if torch.cuda.is_available():
        pytest.skip("the made-up pointers are for a machine without a GPU")
    lib, p = sv._native.load(), ctypes.c_void_p
    INVALID, HIP = 1, 4

    def quantized(L, K=3, acc=0x1000):
        return lib.spec_kv_commit_quantized(None, None, p(0x4000), p(acc), p(0x2000), p(0x3000), None, 2, 4, K, L, 8, 1, None)

    def plain(L, K=3, acc=0x1000):
        return lib.spec_kv_commit(None, p(0x4000), p(acc), p(0x2000), None, 2, 4, K, L, 8, 1, None)
    for f in (quantized, plain):
        assert f(0) == HIP and f(0, K=0) == HIP
        assert f(1) == INVALID and f(0, acc=0x1001) in (INVALID, HIP)


@pytest.mark.gpu
@pytest.mark.parametrize("apart", [True, False])
@pytest.mark.parametrize("K", [0, 1, 40])
def test_commits(apart, K):
    acc = torch.tensor([0, 1, K, -1, 0, K + 1], dtype=torch.int32, device=DEV)
    at = torch.tensor([0, 0, 0, 0, 1, 0], dtype=torch.int32, device=DEV)
    # more than K: 2; a length past the cache, or drafts with no room for them: 1
    want = [2 if not 0 <= n <= K else 1 if a + n > 0 else 0 for n, a in zip(acc.tolist(), at.tolist())]
    staging = torch.randn(3, 6, K, 130, device=DEV)
    codes = torch.empty(3, 6, 0, 130, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    scales = torch.empty(3, 6, 0, 2, dtype=torch.uint8, device=DEV).view(torch.float8_e8m0fnu)
    ln, new = at.clone(), torch.full_like(at, -7) if apart else None
    assert sv.spec_kv_commit_quantized(codes, scales, staging, acc, ln, new_len=new).tolist() == want
    assert (new if apart else ln).tolist() == at.tolist()
    ln = at.clone()
    assert sv.spec_kv_commit(torch.empty(3, 6, 0, 130, device=DEV), staging, acc, ln).tolist() == want
    assert ln.tolist() == at.tolist()


@pytest.mark.gpu
def test_fewer_rows_than_drafts():
    """K beyond L_max: what fits is committed."""
    from tests.test_quantized_rows_and_cache import BF, F32, check_commit
    check_commit(3, 5, 40, 7, 136, BF, [7, 8, 0, 3, 40], [0, 0, 7, 4, 0])
    check_commit(40, 40, 30, 4, 256, F32, [i % 6 for i in range(40)], [i % 5 for i in range(40)])
