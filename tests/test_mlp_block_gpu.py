"""The example block: norm, products, SwiGLU and their backward passes together (GPU).

The bounds come from the formats: an int8 group's codes are within 1/254 of its
largest value, about 1% of a normal value's size, so two chained products of two
such operands stay under 5%.  An E2M1 code is within an eighth of its value for
most values and a block's largest may saturate by a quarter: about 12 to 15% a
operand, a fifth for a product of two, and under 45% for two products in a chain
with the SwiGLU between them.
"""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("T,D,H", [(512, 1024, 1408), (100, 256, 384), (1, 128, 256)])
def test_block(T, D, H):
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    spec = importlib.util.spec_from_file_location("mlp_block", os.path.join(ROOT, "examples", "mlp_block.py"))
    block = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(block)
    errors = block.main(T, D, H)
    print(T, D, H, errors, flush=True)
    for name, err in errors.items():
        assert err < (2.0**-8 if name == "int8 h" else 0.05 if name.startswith("int8") else 0.45), name
