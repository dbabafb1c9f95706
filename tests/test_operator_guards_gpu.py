"""Nothing is written outside the outputs of the norm and microscaled operators (GPU).

Every output lies between two guards of at least 32 of its rows (what a tile or
a block reaches past the last row), filled with a pattern that has to be there
afterwards, and the results are those of outputs with nothing around them.
"""

import numpy as np
import pytest
import torch

import rows64
import swiglu_backward_int8_amd as sq
from test_mxfp4_gpu import check_quant, operands, values
from test_rms_norm_gpu import bwd_inputs, check_backward, check_forward, inputs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
PATTERN = 0xA5


class Guarded:
    """A tensor inside a larger buffer, 256-byte aligned as the allocator's own."""

    def __init__(self, *shape, dtype=torch.uint8):
        size = torch.empty((), dtype=dtype).element_size()
        row = size * (shape[1] if len(shape) > 1 else 1)
        n = size * int(np.prod(shape))
        self.start = -(-max(4096, 32 * row) // 256) * 256
        self.end = self.start + n
        self.room = torch.full((self.end + self.start,), PATTERN, dtype=torch.uint8, device=DEV)
        self.tensor = self.room[self.start:self.end].view(dtype).view(shape)

    def check(self):
        assert bool((self.room[:self.start] == PATTERN).all()), "written in front of the output"
        assert bool((self.room[self.end:] == PATTERN).all()), "written behind the output"


# one row, one row past a block, one short of a block and of a tile; rows of
# codes from 16 bytes to 32 KB; both tile sizes
QUANT = [(1, 1), (1, 9), (2, 8), (1, 70000), (31, 64), (33, 11), (33, 5), (65, 4096), (97, 1000), (127, 520), (129, 264),
         (33, 22016), (161, 30001), (3297, 3848), (3329, 3842), (49153, 9), (49153, 7), (6401, 2048)]


@pytest.mark.parametrize("R,K", QUANT)
def test_quant(R, K):
    x = values(R, K, R + K)
    xd = x.to(DEV)
    for rows, cols in ((True, True), (True, False), (False, True)):
        print("guards of the quantiser", R, K, rows, cols, flush=True)
        out = [Guarded(*s) for s in sq.mxfp4_shapes(R, K)] if rows else [None, None]
        out += [Guarded(*s) for s in sq.mxfp4_shapes(K, R)] if cols else [None, None]
        q, s, qt, st = (None if o is None else o.tensor for o in out)
        sq.mxfp4_quant(xd, q, s, q_t=qt, s_t=st)
        torch.cuda.synchronize()
        for o in out:
            if o is not None:
                o.check()
        if R * K <= 4 << 20:
            check_quant([None if o is None else o.tensor.cpu().numpy() for o in out], x)


@pytest.mark.parametrize("T,D", [(1, 1), (3, 7), (5, 33), (33, 1001), (7, 512), (9, 1024), (4, 2050), (3, 4096), (5, 4097),
                                 (2, 16384), (3, 20001)])
@pytest.mark.parametrize("group,e4m3", [(128, False), (32, True)])
def test_norm(T, D, group, e4m3):
    print("guards of the norm", T, D, group, e4m3, flush=True)
    x, r, w = inputs(T, D, D % 2 == 1, True, seed=T + D)
    q = Guarded(T, D, dtype=torch.uint8 if e4m3 else torch.int8)
    s = Guarded(T, -(-D // group), dtype=torch.float32)
    y, h = Guarded(T, D, dtype=torch.bfloat16), Guarded(T, D, dtype=torch.bfloat16)
    rstd = Guarded(T, dtype=torch.float32)
    sq.rms_norm_quant(x.to(DEV), w.to(DEV), q.tensor, s.tensor, residual=r.to(DEV), h=h.tensor, rstd=rstd.tensor,
                      y_bf16=y.tensor, eps=1e-6, group_size=group)
    torch.cuda.synchronize()
    for o in (q, s, y, h, rstd):
        o.check()
    check_forward(x, r, w, [o.tensor.cpu() for o in (q, s, y, h, rstd)], group, e4m3)


@pytest.mark.parametrize("T,D", [(1, 1), (3, 7), (5, 33), (300, 96), (33, 1001), (700, 520), (4, 2050), (3, 4097), (2, 16384),
                                 (3, 20001), (300, 16640)])
def test_norm_backward(T, D):
    print("guards of the norm's backward pass", T, D, flush=True)
    args = bwd_inputs(T, D, D % 2 == 0, True, seed=T + D)
    dy, h, w, rstd, d_h = (t.to(DEV) for t in args)
    dx, dw = Guarded(T, D, dtype=torch.bfloat16), Guarded(D, dtype=torch.float32)
    ws = Guarded(sq.rms_norm_bwd_workspace(T, D, DEV).numel())
    sq.rms_norm_bwd(dy, h, w, rstd, dx.tensor, dw=dw.tensor, d_h=d_h, workspace=ws.tensor)
    torch.cuda.synchronize()
    for o in (dx, dw, ws):
        o.check()
    check_backward(*args, dx.tensor.cpu(), dw.tensor.cpu())


@pytest.mark.parametrize("R,K", [(1, 1), (3, 7), (5, 33), (64, 128), (33, 1001), (2, 22016), (300, 520), (4201, 1100)])
def test_dequantisers(R, K):
    print("guards of the dequantisers", R, K, flush=True)
    rng = np.random.default_rng(R + K)
    out = Guarded(R, K, dtype=torch.bfloat16)
    (qs, ss) = sq.mxfp4_shapes(R, K)
    q, s = rng.integers(0, 256, qs).astype(np.uint8), rng.integers(100, 150, ss).astype(np.uint8)
    sq.mxfp4_dequant(torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV), out.tensor)
    torch.cuda.synchronize()
    out.check()
    assert np.array_equal(out.tensor.cpu().double().numpy(), rows64.mx_values(q, s)[:, :K])
    for group in (128, 32):
        out = Guarded(R, K, dtype=torch.bfloat16)
        q = rng.integers(-127, 128, (R, K)).astype(np.int8)
        s = rng.random((R, -(-K // group))).astype(np.float32)
        sq.group_dequant(torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV), out.tensor, group_size=group)
        torch.cuda.synchronize()
        out.check()
        want = torch.from_numpy(q.astype(np.float32) * np.repeat(s, group, 1)[:, :K]).bfloat16()
        assert torch.equal(out.tensor.cpu(), want)


# the stream, the slices, and both tiles, with and without whole words of exponents
@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 500, 4096), (20, 9001, 256), (33, 130, 2048), (100, 1001, 1024),
                                   (250, 4001, 640), (777, 1001, 1376), (1401, 2001, 1152), (1500, 2101, 2080), (4353, 4361, 160),
                                   (4353, 4361, 256)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_product(M, N, K, dtype):
    print("guards of the product", M, N, K, dtype, flush=True)
    ops = operands(M, N, K, (126, 127), M + N + K)
    want = rows64.mx_values(*ops[:2]) @ rows64.mx_values(*ops[2:]).T
    C = Guarded(M, N, dtype=dtype)
    sq.mxfp4_gemm(*(torch.from_numpy(t).to(DEV) for t in ops), C.tensor)
    torch.cuda.synchronize()
    C.check()
    assert torch.equal(C.tensor.cpu(), torch.from_numpy(want.astype(np.float32)).to(dtype))
