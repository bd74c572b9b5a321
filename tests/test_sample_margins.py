"""No row of the draws' tests on equal logits, extreme values and very long rows is left out as too near a border:
these tests do not look at how many rows their comparison leaves out, and would pass if it were all of them (CPU)."""
import pytest
import torch

from tests import tree_ref as R
from tests.test_sample_tokens import BF, F32, OFF, logits, near


def left_out(x, u, settings):
    rows = [v if isinstance(v, (list, tuple)) else [v] * len(x) for v in settings]
    values = x.double().numpy()
    return sum(R.sample(values[r], u[r], *(v[r] for v in rows))[1] <= near(x.shape[1]) for r in range(len(x)))


def test_rows_of_two_million():
    x, u = logits(4, 2_000_003, BF, 1, spread=1.0)
    assert left_out(x, u, ([1.0, 1.0, 1.0, 0.0], [0, 3000, 0, 0], [1.0, 1.0, 0.5, 1.0], [0.0, 0.0, 0.0, 0.0])) == 0


@pytest.mark.parametrize("V", [1, 5, 700, 40000])
def test_equal_logits(V):
    x = torch.full((12, V), 2.5)
    x[6:] = torch.randint(0, 3, (6, V), generator=torch.Generator().manual_seed(V))
    for s in (OFF, (1.0, 3, 1.0, 0.0), (1.0, 0, 0.3, 0.0), (1.0, 600, 0.77, 0.0), (0.5, 0, 1.0, 0.9), (0.0, 0, 1.0, 0.0)):
        assert left_out(x, [0.0, 0.3, 0.999999] * 4, s) == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_extreme_temperatures_and_values(dtype):
    x, u = logits(8, 500, dtype, 6)
    big = torch.tensor(torch.finfo(dtype).max)
    for T in (1e-45, 1e-30, 1e-3, 1e4, 1e30, 3e38):
        assert left_out(x, u, (T, 0, 0.9, 0.0)) == 0
        assert left_out((x / x.abs().max() * big).to(dtype), u, (T, 30, 1.0, 0.2)) == 0
    x[:, 3] = big.to(dtype)
    x[:, 4] = -big.to(dtype)
    assert left_out(x, u, (1.0, 0, 1.0, 0.0)) == 0
