"""Rows of the layer norm whose offset is so many standard deviations that offset
times rstd passes fp32's range (GPU).  A place past a row's end holds no element: it
may not reach the row's codes, scales or gradients.

The rows are of one value 2^100, whose sums and mean fp32 holds exactly, with eps
1e-20, so rstd = 1e10: (h - mean) * rstd is 0 everywhere in the row, y is the bias,
and dx is rstd * (g - sum(g) / D) + d_h.  That is a sum of D products of fp32 numbers
and their mean taken from each: (L + 4) u of the magnitudes, with u = 2^-24 and L the
longest chain of additions as for the other rows, and half a step of bf16.
"""

import numpy as np
import pytest
import torch

import ln64
import rows64
from test_layer_norm_gpu import BF16_HALF_ULP, RNG, U, chain, run_backward, run_forward

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


@pytest.mark.parametrize("T,D", [(3, D) for D in WIDTHS] + [(700, 200), (700, 1001), (300, 4100)])
@pytest.mark.parametrize("dy32", [False, True])
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_gradients(T, D, dy32, p):
    g = torch.Generator().manual_seed(D)
    h = torch.full((T, D), VALUE).bfloat16()
    w = (1 + 0.3 * torch.randn(D, generator=g)).bfloat16()
    dy = torch.randn(T, D, generator=g) * 0.01
    dy = dy if dy32 else dy.bfloat16()
    d_h = (torch.randn(T, D, generator=g) * 1e7).bfloat16()
    mean, rstd = torch.full((T,), VALUE), torch.full((T,), 1e10)
    dx, drop, dw, db = run_backward(dy, h, w, mean, rstd, d_h, p=p)
    gr = dy.double() * w.double()
    want = 1e10 * (gr - gr.mean(1, keepdim=True)) + d_h.double()
    err = (chain(D) + 4) * U * (1e10 * (gr.abs() + gr.abs().mean(1, keepdim=True)) + d_h.double().abs())
    assert ((dx.double() - want).abs() <= BF16_HALF_ULP * 1.001 * want.abs() + err).all()
    if p > 0:
        keep, scale = ln64.kept(RNG, T, D, p), ln64.scale(p)
        assert (drop[~keep] == 0).all()
        assert ((drop.double() - scale * want).abs() <= scale * ((BF16_HALF_ULP + U) * 1.001 * want.abs() + err))[keep].all()
    assert (dw == 0).all()
    assert ((db.double() - dy.double().sum(0)).abs() <= (T + 32) * U * dy.double().abs().sum(0)).all()
