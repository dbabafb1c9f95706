"""Nothing is written outside the outputs of the layer norm, the dropout and the gated
projection, and nothing outside the inputs reaches them (GPU).

Every output lies between two guards of at least 32 of its rows filled with a
pattern that has to be there afterwards; the inputs lie between rows of NaN, so
that a value read past them would show.
"""

import numpy as np
import pytest
import torch

import ln64
import swiglu_backward_int8_amd as sq
from test_layer_norm_gpu import RNG, bwd_inputs, check_backward, check_forward, inputs, rng_tensor
from test_operator_guards_gpu import DEV, Guarded
from test_swiglu_gemm_gpu import check_d_gu, check_products, normal, silu, whole

pytestmark = pytest.mark.gpu

bf16, f32 = torch.bfloat16, torch.float32


def fenced(t):
    """t on the GPU between 64 of its rows (at least 4 KB) of NaN on either side, 256-byte aligned."""
    size = t.element_size()
    row = size * (t.shape[1] if t.dim() > 1 else 1)
    side = -(-max(4096, 64 * row) // 256) * 256
    room = torch.full(((2 * side + size * t.numel()) // size,), float("nan"), dtype=t.dtype, device=DEV)
    at = side // size
    out = room[at:at + t.numel()].view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("T,D", [(1, 1), (3, 7), (5, 33), (33, 1001), (7, 512), (9, 1024), (4, 2050), (3, 4096), (5, 4097), (3, 9001),
                                 (2, 16384), (3, 20001)])
@pytest.mark.parametrize("group,e4m3,p", [(128, False, 0.0), (32, True, 0.3)])
def test_norm(T, D, group, e4m3, p):
    print("guards of the norm", T, D, group, e4m3, p, flush=True)
    x, r, w, b = inputs(T, D, D % 2 == 1, True, seed=T + D)
    q = Guarded(T, D, dtype=torch.uint8 if e4m3 else torch.int8)
    s = Guarded(T, -(-D // group), dtype=f32)
    y, h = Guarded(T, D, dtype=bf16), Guarded(T, D, dtype=bf16)
    mean, rstd = Guarded(T, dtype=f32), Guarded(T, dtype=f32)
    outs = (q, s, y, h, mean, rstd)
    sq.layer_norm_quant(fenced(x), fenced(w), fenced(b), q.tensor, s.tensor, residual=fenced(r), h=h.tensor, mean=mean.tensor,
                        rstd=rstd.tensor, y_bf16=y.tensor, group_size=group, p=p, rng=rng_tensor())
    torch.cuda.synchronize()
    for o in outs:
        o.check()
    check_forward(x, r, w, b, [o.tensor.cpu() for o in outs], group, e4m3, p=p)


@pytest.mark.parametrize("T,D", [(1, 1), (3, 7), (5, 33), (300, 96), (33, 1001), (700, 520), (4, 2050), (3, 4097), (40, 9001),
                                 (2, 16384), (3, 20001), (300, 16640)])
def test_norm_backward(T, D):
    print("guards of the norm's backward pass", T, D, flush=True)
    args = bwd_inputs(T, D, D % 2 == 0, True, seed=T + D)
    dx, drop = Guarded(T, D, dtype=bf16), Guarded(T, D, dtype=bf16)
    dw, db = Guarded(D, dtype=f32), Guarded(D, dtype=f32)
    ws = Guarded(sq.layer_norm_bwd_workspace(T, D, DEV).numel())
    dy, h, w, mean, rstd, d_h = (fenced(t) for t in args)
    sq.layer_norm_bwd(dy, h, w, mean, rstd, dx.tensor, dw=dw.tensor, db=db.tensor, d_h=d_h, dx_drop=drop.tensor, workspace=ws.tensor,
                      p=0.2, rng=rng_tensor())
    torch.cuda.synchronize()
    for o in (dx, drop, dw, db, ws):
        o.check()
    check_backward(*args, [o.tensor.cpu() for o in (dx, drop, dw, db)], p=0.2)


@pytest.mark.parametrize("T,D", [(1, 1), (3, 7), (5, 33), (33, 1001), (7, 512), (64, 4096), (3, 11008), (2, 70001)])
@pytest.mark.parametrize("x32", [False, True])
def test_dropout(T, D, x32):
    print("guards of the dropout", T, D, x32, flush=True)
    x, r, _, _ = inputs(T, D, x32, True, seed=T + D)
    out = Guarded(T, D, dtype=bf16)
    sq.dropout_add(fenced(x), out.tensor, 0.4, rng_tensor(), residual=fenced(r))
    torch.cuda.synchronize()
    out.check()
    assert torch.equal(out.tensor.cpu().view(torch.int16), ln64.stream(x, r, 0.4, RNG).view(torch.int16))


# the stream, all four tiles, whole and not, with and without a last part of K
SHAPES = [(1, 8, 8), (3, 520, 264), (16, 1000, 1032), (20, 72, 72), (70, 264, 136), (130, 1000, 392), (300, 520, 520),
          (1100, 1032, 264), (2050, 4104, 328), (513, 8200, 72)]


@pytest.mark.parametrize("T,H,D", SHAPES)
@pytest.mark.parametrize("keep", [False, True])
def test_projection(T, H, D, keep):
    print("guards of the projection", T, H, D, keep, flush=True)
    x, w = whole(T, H, D, T + H + D)
    y, gu = Guarded(T, H, dtype=bf16), Guarded(T, 2 * H, dtype=bf16) if keep else None
    sq.swiglu_gemm(fenced(x), fenced(w), y.tensor, gu=gu.tensor if keep else None)
    torch.cuda.synchronize()
    y.check()
    want = x.double() @ w.double().t()
    if keep:
        gu.check()
        assert torch.equal(gu.tensor, want.to(bf16))
    gate, up = want.chunk(2, 1)
    v = silu(gate) * up
    assert ((y.tensor.double() - v).abs() <= 2.0**-8 * 1.001 * v.abs() + 4 * (gate.abs() + 4) * 2.0**-24 * v.abs() + 1e-38).all()


# the same with long sums over few tiles, which are taken in slices
@pytest.mark.parametrize("T,H,D", SHAPES + [(40, 8200, 200), (300, 11008, 264), (9000, 72, 104)])
@pytest.mark.parametrize("dtype", [bf16, f32])
def test_projection_backward(T, H, D, dtype):
    print("guards of the projection's backward pass", T, H, D, dtype, flush=True)
    x, w = normal(T, H, D, T + H + D)
    g = torch.Generator(device=DEV).manual_seed(T)
    gu = (torch.randn((T, 2 * H), generator=g, device=DEV) * 2).to(bf16)
    dy = (torch.randn((T, H), generator=g, device=DEV) * 0.01).to(bf16)
    d_gu = Guarded(T, 2 * H, dtype=bf16)
    dx, dw = Guarded(T, D, dtype=dtype), Guarded(2 * H, D, dtype=dtype)
    ws = Guarded(sq.swiglu_gemm_bwd_workspace(T, H, D, DEV).numel())
    ws.tensor.fill_(0xff)  # NaN
    sq.swiglu_gemm_bwd(fenced(dy), fenced(gu), fenced(x), fenced(w), d_gu.tensor, dx=dx.tensor, dw=dw.tensor, workspace=ws.tensor)
    torch.cuda.synchronize()
    for o in (d_gu, dx, dw, ws):
        o.check()
    check_d_gu(d_gu.tensor, dy, gu)
    check_products(d_gu.tensor, x, w, dx.tensor, dw.tensor)


def test_the_last_rows_of_slices_meet():
    # K that no slice count divides: the last slice is short, and some counts leave slices with nothing
    for K in (64 * 17, 64 * 33, 64 * 45 + 8, 64 * 172):
        T, H, D = 24, K // 2 // 8 * 8, 72
        x, w = whole(T, H, D, K)
        dy = torch.ones((T, H), device=DEV).to(bf16)
        gu = torch.cat([torch.zeros((T, H), device=DEV), torch.randint(-2, 3, (T, H), device=DEV).float()], 1).to(bf16)
        d_gu, dx = torch.empty((T, 2 * H), dtype=bf16, device=DEV), torch.empty((T, D), dtype=f32, device=DEV)
        sq.swiglu_gemm_bwd(dy, gu, x, w, d_gu, dx=dx, workspace=sq.swiglu_gemm_bwd_workspace(T, H, D, DEV))
        assert torch.equal(dx.double(), d_gu.double() @ w.double())
    assert np.isfinite(float(dx.sum()))
