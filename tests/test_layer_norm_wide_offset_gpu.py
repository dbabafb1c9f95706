"""Rows of more than 16384 columns whose offset's square passes fp32's range, while
the squares of the differences do not (GPU).  Bounds as for the other rows."""

import pytest
import torch

from test_layer_norm_gpu import check_forward, run_forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [16384, 16385, 16392, 20001, 32768, 70001])
@pytest.mark.parametrize("power", [40, 63, 65])
def test_statistics(D, power):
    # one value in 128 is a step of bf16 higher: a variance of 2^(2 power - 14) / 128, sums of squares below 2^(2 power - 4)
    g = torch.Generator().manual_seed(D)
    x = torch.full((4, D), 2.0**power)
    x[torch.rand((4, D), generator=g) < 1 / 128] *= 1 + 2.0**-7
    x[1], x[3] = -x[1], 0.0
    x = x.bfloat16()
    w, b = (1 + 0.3 * torch.randn(D, generator=g)).bfloat16(), torch.randn(D, generator=g).bfloat16()
    out = run_forward(x, None, w, b, 128, False)
    assert all(torch.isfinite(t.float()).all() for t in out)
    check_forward(x, None, w, b, out, 128, False)
