"""The microscaled product's tiles of a few rows or columns, in front of others that the
same workgroup takes next (GPU): most of its waves have nothing to store there.  Sums
that fp32 holds exactly, equal to the last bit, several times each, since what one wave
leaves to another depends on their timing."""

import pytest
import torch

import rows64
import swiglu_backward_int8_amd as sq
from test_mxfp4_gpu import DEV, operands

pytestmark = pytest.mark.gpu

# 128 x 128: more than 512 tiles, that 256 x 256 would take in more time; 256 x 256: more than 256
SHAPES = [(40, 131000, 128), (40, 131000, 640), (261, 43500, 128), (261, 43500, 640), (261, 43500, 1184), (4357, 4360, 128),
          (4357, 4360, 640), (4357, 4360, 1184), (4360, 4357, 768), (6661, 4101, 96)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_products(M, N, K):
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    print("product", M, N, K, flush=True)
    ops = operands(M, N, K, (126, 127), M + N + K)
    a, b = (torch.from_numpy(rows64.mx_values(*o)).to(DEV) for o in (ops[:2], ops[2:]))
    want = a @ b.t()
    on_gpu = [torch.from_numpy(t).to(DEV) for t in ops]
    for i in range(6):
        for dtype in (torch.float32, torch.bfloat16):
            C = torch.full((M, N), float("nan"), dtype=dtype, device=DEV)
            sq.mxfp4_gemm(*on_gpu, C)
            assert torch.equal(C, want.to(dtype)), (i, dtype)
