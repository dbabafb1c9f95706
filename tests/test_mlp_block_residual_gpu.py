"""The residual's gradient in the example block (GPU): d_h reaches d_x whole, and nothing else.

d_x = bf16(A + d_h) with an A that does not depend on d_h, so two runs that
differ in d_h alone differ by it, up to the rounding of either d_x: half an ulp,
2^-8 of its magnitude at most (and what the fp32 sum adds, below 1% of that).
"""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("T,D,H", [(512, 1024, 1408), (100, 256, 384), (1, 128, 256)])
def test_residual_gradient(T, D, H):
    spec = importlib.util.spec_from_file_location("mlp_block", os.path.join(ROOT, "examples", "mlp_block.py"))
    block = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(block)
    dev = "cuda:0"
    g = torch.Generator(device=dev).manual_seed(1)
    rand = lambda *shape, std=1.0: (torch.randn(shape, generator=g, device=dev) * std).bfloat16()
    x, residual, w = rand(T, D), rand(T, D), (1 + rand(D, std=0.1).float()).bfloat16()
    Wgu, Wd = rand(2 * H, D, std=D**-0.5), rand(D, H, std=H**-0.5)
    d_out, d_h = rand(T, D, std=0.01), rand(T, D, std=0.01)
    args = x, residual, w, Wgu, Wd, d_out
    out, d_x, *rest = block.train_mxfp4(*args, d_h)
    out0, d_x0, *rest0 = block.train_mxfp4(*args, torch.zeros_like(d_h))
    for a, b in zip([out] + rest, [out0] + rest0):
        assert torch.equal(a, b)
    a, b, d = d_x.double(), d_x0.double(), d_h.double()
    assert ((a - b - d).abs() <= 1.01 * 2.0**-8 * (a.abs() + b.abs()) + 1e-40).all()
    assert ((a - b).abs() > 0).sum() > 0.9 * d.numel()  # the bound is below d_h nearly everywhere
