"""What the operators of a step with a tree of drafts refuse, beside their own tests (CPU)."""
import pytest

from tests import test_sample_tokens as sample
from tests import test_tree_attention as attention
from tests import test_tree_commit as commit

OK, INVALID, WORKSPACE = 0, 1, 3


@pytest.mark.parametrize("quantized", [False, True])
def test_scales_that_overflow_in_the_exponents_base(quantized):
    """The largest scales are finite themselves, but not times log2(e), which every score is multiplied by."""
    assert attention.c_call(quantized, scale=2.35e38) == WORKSPACE   # valid, but for the workspace
    for scale in (2.37e38, 3.4e38):
        assert attention.c_call(quantized, scale=scale) == INVALID


# ---- outputs that overlap other buffers ------------------------------------------
# Calls are refused before anything is launched, so that made-up addresses do; those that are taken run on a GPU.

def spans(sizes, start=1 << 40):
    """Addresses, 256 bytes apart at least, of buffers of these sizes."""
    at = {}
    for name, size in sizes.items():
        at[name] = start
        start += (size + 511) // 256 * 256
    return at


def attention_sizes(quantized, dt, B=2, N=3, Hq=4, Hkv=2, D=64, L=5000):
    es = 2 if dt == 1 else 4
    cache = B * L * Hkv * D * (1 if quantized else es)
    sizes = dict(q=B * N * Hq * D * es, k=cache, v=cache, kn=B * N * Hkv * D * es, vn=B * N * Hkv * D * es,
                 par=B * N * 4, n=B * 4, out=B * N * Hq * D * es,
                 ws=attention.sv()._native.load().spec_tree_attention_workspace_bytes(B, N, Hq, Hkv, D, L, dt))
    if quantized:
        sizes.update(ks=B * L, vs=B * L)
    return sizes


@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("dt", [0, 1])
def test_attention_refuses_outputs_over_other_buffers(quantized, dt):
    """The output's first and last byte in another buffer, and the workspace's."""
    sizes = attention_sizes(quantized, dt)
    at = spans(sizes)
    es = 2 if dt == 1 else 4

    def call(**over):
        return attention.c_call(quantized, dt=dt, wsb=sizes["ws"], **{**at, **over})
    for name in at:
        if name in ("out", "ws"):
            continue
        end = at[name] + sizes[name]
        assert call(out=end - 4) == INVALID, name                                    # the output's beginning
        assert call(out=at[name] - sizes["out"] + 4) == INVALID, name                # its end
        ws = (end - 1) // 256 * 256
        assert call(ws=ws) == INVALID, name
        assert call(ws=(at[name] - sizes["ws"]) // 256 * 256 + 256) == INVALID, name
    assert call(out=at["q"] + es) == INVALID and call(out=at["q"] - es) == INVALID   # not the queries themselves
    assert call(out=at["q"], kn=at["q"]) == INVALID                                  # those alone
    assert call(out=at["ws"]) == INVALID


@pytest.mark.parametrize("dt", [0, 1])
def test_sampling_refuses_tokens_over_its_inputs(dt):
    R, V = 5, 130
    sizes = dict(x=R * V * (2 if dt == 1 else 4), u=R * 4, T=R * 4, k=R * 4, p=R * 4, m=R * 4, out=R * 4)
    at = spans(sizes)
    for name in ("x", "u", "T", "k", "p", "m"):
        for out in (at[name], at[name] + sizes[name] - 4, at[name] - sizes["out"] + 4):
            assert sample.c_call(R=R, V=V, dt=dt, **{**at, "out": out}) == INVALID, name


@pytest.mark.parametrize("quantized", [False, True])
@pytest.mark.parametrize("dt", [0, 1])
def test_commits_refuse_a_cache_or_staging_over_other_buffers(quantized, dt):
    P, B, N, L, E = 2, 3, 4, 16, 64
    es = 2 if dt == 1 else 4
    sizes = dict(cache=P * B * L * E * (1 if quantized else es), scales=P * B * L, staging=P * B * N * E * es,
                 tok=B * N * 4, par=B * N * 4, sam=B * N * 4, n=B * 4, new=B * 4, acc=B * 4, out=B * N * 4, path=B * N * 4,
                 st=B * 4)
    assert set(sizes) == set(commit.FAR)
    at = spans(sizes)

    def call(**over):
        return commit.c_call(quantized, dt=dt, P=P, B=B, N=N, L=L, E=E, **{**at, **over})
    lists = [n for n in sizes if n not in ("cache", "scales", "staging")]
    for buf in ["cache", "staging"] + ["scales"] * quantized:
        for name in lists:
            if buf == "staging" and name in ("tok", "par", "sam", "n"):
                continue                                                       # it is read alone, as they are
            for x in (at[name] + sizes[name] - 4, at[name] - sizes[buf] + 4):
                assert call(**{buf: x}) == INVALID, (buf, name)
    for a, b in [("cache", "staging")] + [("scales", "staging"), ("cache", "scales")] * quantized:
        assert call(**{a: at[b] + sizes[b] - 4}) == INVALID and call(**{a: at[b] - sizes[a] + 4}) == INVALID
