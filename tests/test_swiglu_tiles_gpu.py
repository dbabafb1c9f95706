"""The gated projection at the sizes of tile_shapes: kernels that the other tests'
sizes leave out, compared as those are, in full, and between guards (GPU)."""

import pytest
import torch

import test_block_guards_gpu as guards
import test_swiglu_gemm_gpu as gemm
import tile_shapes

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    gemm.sq.lib()
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,H,D", tile_shapes.SHAPES)
def test_forward(T, H, D):
    gemm.test_forward(T, H, D)


@pytest.mark.parametrize("T,H,D", tile_shapes.SHAPES)
def test_backward(T, H, D):
    gemm.test_backward(T, H, D)


@pytest.mark.parametrize("T,H,D", tile_shapes.SHAPES)
@pytest.mark.parametrize("keep", [False, True])
def test_guards_of_the_forward_pass(T, H, D, keep):
    guards.test_projection(T, H, D, keep)


@pytest.mark.parametrize("T,H,D", tile_shapes.SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_guards_of_the_backward_pass(T, H, D, dtype):
    guards.test_projection_backward(T, H, D, dtype)
