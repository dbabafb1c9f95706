"""Gates so far below zero that silu(gate) alone is a denormal number of fp32 or 0, and
up so large that y is not (GPU).  y is within half a step of bf16 and 4 (|gate| + 4) u
of the formula, as everywhere; u = 2^-24."""

import pytest
import torch

import swiglu_backward_int8_amd as sq
from test_swiglu_gemm_gpu import DEV, HALF, U, run_forward, silu

pytestmark = pytest.mark.gpu


# the streams and tiles of every size
@pytest.mark.parametrize("T,H,D", [(1, 104, 8), (20, 104, 8), (40, 104, 8), (65, 104, 72), (4097, 520, 72), (3501, 3512, 216), (2632, 3096, 592)])
def test_y_keeps_the_bits_of_small_gates(T, H, D):
    sq.lib()
    gates = torch.linspace(-150, -80, 8 * 13, device=DEV).repeat(-(-H // 104))[:H]
    ups = 2.0 ** torch.linspace(60, 120, 8 * 13, device=DEV).flip(0).repeat(-(-H // 104))[:H]  # the lower the gate, the larger
    x = torch.zeros((T, D), device=DEV)
    x[:, 0] = 1.0
    w = torch.zeros((2 * H, D), device=DEV)
    w[:H, 0], w[H:, 0] = gates, ups
    x, w = x.bfloat16(), w.bfloat16()
    y, gu = run_forward(x, w)
    gate, up = w[:H, 0].double(), w[H:, 0].double()
    assert torch.equal(gu[-1].double(), torch.cat([gate, up]))
    want = silu(gate) * up
    assert (want.abs() > 2.0**-120).all() and (silu(gate).abs() < 2.0**-126).sum() > H // 2
    assert ((y.double() - want).abs() <= HALF * 1.001 * want.abs() + 4 * (gate.abs() + 4) * U * want.abs()).all()
