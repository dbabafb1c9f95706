"""Rows of the layer norm whose offset is so many standard deviations that offset
times rstd passes fp32's range (GPU).  A place past a row's end holds no element: it
may not reach the row's codes and scales.

The rows are of one value 2^100, whose sums and mean fp32 holds exactly, with eps
1e-20, so rstd = 1e10: (h - mean) * rstd is 0 everywhere in the row and y the bias.
"""

import numpy as np
import pytest
import torch

import ln64
import rows64
from test_layer_norm_gpu import RNG, U, run_forward

pytestmark = pytest.mark.gpu

VALUE, EPS = 2.0**100, 1e-20
# rows off 16 bytes and of whole pieces, of a wave, of a workgroup and walked twice
WIDTHS = [1, 5, 9, 64, 200, 513, 520, 1001, 1032, 2050, 4096, 4100, 9001, 16392, 17001]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("group,e4m3,p", [(128, False, 0.0), (32, True, 0.0), (64, False, 0.25)])
def test_codes(D, group, e4m3, p):
    g = torch.Generator().manual_seed(D)
    w, b = (1 + 0.3 * torch.randn(D, generator=g)).bfloat16(), (0.2 * torch.randn(D, generator=g)).bfloat16()
    if p == 0:
        x, r = torch.full((3, D), VALUE).bfloat16(), None
    else:  # what is dropped comes back through the residual
        keep = ln64.kept(RNG, 3, D, p)
        x, r = torch.full((3, D), 0.0).bfloat16(), torch.full((3, D), VALUE).bfloat16()
        x = torch.where(keep, x, torch.tensor(float("inf")).bfloat16())
    q, s, y, h, mean, rstd = run_forward(x, r, w, b, group, e4m3, eps=EPS, p=p)
    assert (h.double() == VALUE).all() and (mean.double() == VALUE).all()
    assert ((rstd.double() - 1e10).abs() <= 4 * U * 1e10).all()
    assert torch.equal(y, b.expand(3, D))
    codes, scales = rows64.group_quant(y, group, e4m3)
    assert np.isfinite(scales).all() and np.array_equal(s.numpy(), scales)
    assert np.array_equal(q.view(torch.uint8).numpy(), codes)
