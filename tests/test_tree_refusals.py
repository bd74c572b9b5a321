"""What the operators of a step with a tree of drafts refuse, beside their own tests (CPU)."""
import pytest

from tests import test_tree_attention as attention

OK, INVALID, WORKSPACE = 0, 1, 3


@pytest.mark.parametrize("quantized", [False, True])
def test_scales_that_overflow_in_the_exponents_base(quantized):
    """The largest scales are finite themselves, but not times log2(e), which every score is multiplied by."""
    assert attention.c_call(quantized, scale=2.35e38) == WORKSPACE   # valid, but for the workspace
    for scale in (2.37e38, 3.4e38):
        assert attention.c_call(quantized, scale=scale) == INVALID
