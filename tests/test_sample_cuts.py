"""Cuts by min-p that fall between the values a row's table tells apart: beside zero, nearer to it than any
value of the table, where zeros are above the cut or below it but never its ties."""
import math

import numpy as np
import pytest
import torch

from tests.test_sample_tokens import BF, DEV, check, sv

# Largest logit, cut, and a temperature and min-p (floats) with which the least float at or above
# largest + T log(min_p) is the cut, a bf16 value of less than 2^-20.
CUTS = [(1.0, 2.0 ** -21, "0x1.57ab34p-2", "0x1.a041a6p-5"), (1.0, -2.0 ** -22, "0x1.d8b462p-1", "0x1.5aa8cep-2"),
        (0.0, -2.0 ** -21, "0x1.254bccp-20", "0x1.4aedf8p-1"), (0.0, -2.0 ** -24, "0x1.254bccp-23", "0x1.4aedf8p-1")]


def settings(cut):
    return float.fromhex(CUTS[cut][2]), float.fromhex(CUTS[cut][3])


@pytest.mark.parametrize("cut", range(len(CUTS)))
def test_the_cut_is_where_it_is_meant_to_be(cut):
    """Whichever way a logarithm good to two units in its last place is rounded."""
    top, at = CUTS[cut][:2]
    T, m = settings(cut)
    for off in (-2.0 ** -52, 0.0, 2.0 ** -52):
        least = top + T * np.log(np.float64(np.float32(m))) * (1 + off)
        f = np.float32(least)
        f = f if float(f) >= least else np.nextafter(f, np.float32(np.inf))
        assert float(f) == at and float(torch.tensor(at).to(BF)) == at


@pytest.mark.gpu
@pytest.mark.parametrize("cut", range(len(CUTS)))
@pytest.mark.parametrize("rows", [16, 300])
def test_a_min_p_cut_beside_zero(cut, rows):
    """Many zeros of both signs and as many tokens above the top-p cut as a draw by table is made for."""
    V = 4096
    top = CUTS[cut][0]
    g = torch.Generator().manual_seed(cut)
    x = torch.full((rows, V), -3.0)
    x[torch.rand((rows, V), generator=g) < 0.25] = 0.0
    x[torch.rand((rows, V), generator=g) < 0.25] = -0.0
    if top > 0:
        x[torch.rand((rows, V), generator=g) < 0.1] = 0.5
        x[torch.rand((rows, V), generator=g) < 0.1] = top
    T, m = settings(cut)
    u = torch.linspace(0, 1, rows + 1)[:-1].tolist()
    got = sv().spec_sample_tokens(x.to(BF).to(DEV), torch.tensor(u, device=DEV), T, top_p=0.999, min_p=m).cpu()
    assert bool((x[torch.arange(rows), got.long()] >= CUTS[cut][1]).all())
    close = check(x.to(BF), u, (T, 0, 0.999, m), got)
    if top > 0:
        assert close <= rows // 100
        return
    # Zeros alone are kept, of one weight: the first ceil(p n) of n by id, and u = i / 16 is a border of such a draw
    # for many i, whose rows the plain draw leaves out.  But products of p or u (24 bits) with a count (12 bits) are
    # exact in 64, so it is token floor(u kept).
    for r in range(rows):
        zeros = (x[r] == 0).nonzero().flatten()
        kept = math.ceil(float(np.float32(0.999)) * len(zeros))
        assert int(got[r]) == int(zeros[int(float(np.float32(u[r])) * kept)])
