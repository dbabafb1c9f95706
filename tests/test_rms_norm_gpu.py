"""The RMS norm with its quantised output, and its backward pass (GPU).

Bounds, with u = 2^-24 and a row's longest chain of additions L = 8 ceil(D /
512) + 32 (a lane's elements, then the joins):
* h is one fp32 addition rounded to bf16: equal bits.
* rstd: the sum of squares is off by at most L u of itself, half of that after
  the root, and division, eps, root and inverse add a rounding each.
* y before rounding is off by rstd's error and two roundings, and the rounding
  to bf16 adds at most 2^-8 of its magnitude (half a unit in the last place).
* codes and scales are those of the kernel's own y_bf16, bit for bit.
* dx: L + 8 roundings of the magnitudes it is made of, and half an ulp of bf16.
* dw: T + 32 roundings of the sum of its terms' magnitudes.
"""

import numpy as np
import pytest
import torch

import rows64
import swiglu_backward_int8_amd as sq

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0**-24
BF16_HALF_ULP = 2.0**-8
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    sq.lib()


def inputs(T, D, x32, residual, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, D, generator=g) * torch.exp(torch.randn(T, 1, generator=g))
    x[:, ::37] *= 30.0
    x[5::11] = 0
    r = torch.randn(T, D, generator=g).bfloat16() if residual else None
    if residual:
        r[5::11] = 0
    w = (1 + 0.3 * torch.randn(D, generator=g)).bfloat16()
    return (x if x32 else x.bfloat16()), r, w


def chain(D):
    return 8 * -(-D // 512) + 32


def run_forward(x, r, w, group, e4m3, y_q=True, y_bf16=True, eps=EPS, inplace=False):
    T, D = x.shape
    q = torch.full((T, D), 55, dtype=torch.uint8 if e4m3 else torch.int8, device=DEV) if y_q else None
    s = torch.full((T, -(-D // group)), float("nan"), device=DEV) if y_q else None
    y = torch.full((T, D), float("nan"), dtype=torch.bfloat16, device=DEV) if y_bf16 else None
    rd = None if r is None else r.to(DEV)
    h = rd if inplace else torch.full((T, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    rstd = torch.full((T,), float("nan"), device=DEV)
    sq.rms_norm_quant(x.to(DEV), w.to(DEV), q, s, residual=rd, h=h, rstd=rstd, y_bf16=y, eps=eps, group_size=group)
    torch.cuda.synchronize()
    return [None if t is None else t.cpu() for t in (q, s, y, h, rstd)]


def check_forward(x, r, w, out, group, e4m3, eps=EPS):
    q, s, y, h, rstd = out
    D = x.shape[1]
    h64, rstd64, y64 = rows64.norm(x, r, w, eps)
    assert torch.equal(h.view(torch.int16), h64.view(torch.int16))
    rel = (chain(D) / 2 + 5) * U
    assert ((rstd.double() - rstd64).abs() <= rel * rstd64).all()
    if y is not None:
        bound = (BF16_HALF_ULP * 1.001 + rel + 3 * U) * y64.abs() + 1e-40
        assert ((y.double() - y64).abs() <= bound).all()
    if q is not None and y is not None:
        codes, scales = rows64.group_quant(y, group, e4m3)
        assert np.array_equal(q.view(torch.uint8).numpy(), codes)
        assert np.array_equal(s.numpy(), scales)


SHAPES = [(1, 1), (1, 4096), (3, 7), (2, 31), (5, 32), (4, 33), (7, 128), (9, 200), (6, 511), (6, 512), (5, 513),
          (33, 1001), (20, 1024), (3, 1376), (4, 2048), (3, 2050), (5, 4095), (2, 4096), (3, 4097), (2, 8192), (3, 8200),
          (2, 11008), (1, 16384), (2, 16385), (2, 22016), (1, 70001)]


@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("group,e4m3", [(128, False), (64, True), (32, False), (32, True)])
def test_forward(T, D, group, e4m3):
    x, r, w = inputs(T, D, x32=(T + D) % 2 == 1, residual=D % 3 != 0, seed=T * 7 + D)
    print("forward", T, D, group, e4m3, flush=True)
    check_forward(x, r, w, run_forward(x, r, w, group, e4m3), group, e4m3)


@pytest.mark.parametrize("T,D", [(2500, 1376), (2304, 4096), (2060, 1001), (4097, 512), (2049, 96), (2111, 2048)])
def test_forward_many_rows(T, D):
    # enough rows for a wave each
    for x32, e4m3 in ((False, False), (True, True)):
        x, r, w = inputs(T, D, x32, True, seed=D)
        check_forward(x, r, w, run_forward(x, r, w, 128, e4m3), 128, e4m3)


@pytest.mark.parametrize("D", [257, 4096, 20000])
def test_forward_in_place_and_optional_outputs(D):
    x, r, w = inputs(4, D, False, True, seed=1)
    full = run_forward(x, r, w, 64, False)
    inplace = run_forward(x, r, w, 64, False, inplace=True)
    for a, b in zip(full, inplace):
        assert torch.equal(a, b)
    only_y = run_forward(x, r, w, 64, False, y_q=False)
    only_q = run_forward(x, r, w, 64, False, y_bf16=False)
    assert torch.equal(only_y[2], full[2]) and torch.equal(only_q[0], full[0]) and torch.equal(only_q[1], full[1])
    # without h and rstd
    q, s = torch.empty_like(full[0], device=DEV), torch.empty_like(full[1], device=DEV)
    sq.rms_norm_quant(x.to(DEV), w.to(DEV), q, s, residual=r.to(DEV), eps=EPS, group_size=64)
    assert torch.equal(q.cpu(), full[0]) and torch.equal(s.cpu(), full[1])


@pytest.mark.parametrize("e4m3", [False, True])
def test_forward_tiny_values_and_zero_eps(e4m3):
    # y down to bf16 subnormals, where the inverse scale overflows: weights of 2^-125 and below
    g = torch.Generator().manual_seed(3)
    x = torch.randn(6, 384, generator=g).bfloat16()
    w = torch.full((384,), 2.0**-126).bfloat16()
    w[128:256] = 2.0**-133
    w[256:] = 2.0**-121
    out = run_forward(x, None, w, 128, e4m3, eps=0.0)
    codes, scales = rows64.group_quant(out[2], 128, e4m3)
    assert np.array_equal(out[0].view(torch.uint8).numpy(), codes) and np.array_equal(out[1].numpy(), scales)


def test_forward_large_values_do_not_overflow_a_row_nearby():
    # an infinity or a NaN stays in its row, and shows in the scales there
    x, r, w = inputs(5, 640, False, True, seed=4)
    want = run_forward(x, r, w, 128, False)
    for bad in (float("inf"), float("nan")):
        y = x.clone()
        y[2, 300] = bad
        got = run_forward(y, r, w, 128, False)
        for a, b in zip(got, want):
            assert torch.equal(a[[0, 1, 3, 4]], b[[0, 1, 3, 4]])
        assert torch.isnan(got[1][2, 2])


def run_backward(dy, h, w, rstd, d_h, want_dw=True, inplace=False):
    T, D = h.shape
    dd = None if d_h is None else d_h.to(DEV)
    dx = dd if inplace else torch.full((T, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    dw = torch.full((D,), float("nan"), device=DEV) if want_dw else None
    ws = sq.rms_norm_bwd_workspace(T, D, DEV).fill_(0xff) if want_dw or D > 16384 else None
    sq.rms_norm_bwd(dy.to(DEV), h.to(DEV), w.to(DEV), rstd.to(DEV), dx, dw=dw, d_h=dd, workspace=ws)
    torch.cuda.synchronize()
    return dx.cpu(), None if dw is None else dw.cpu()


def bwd_inputs(T, D, dy32, with_d_h, seed):
    g = torch.Generator().manual_seed(seed)
    h = (torch.randn(T, D, generator=g) * torch.exp(torch.randn(T, 1, generator=g))).bfloat16()
    w = (1 + 0.3 * torch.randn(D, generator=g)).bfloat16()
    rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
    dy = torch.randn(T, D, generator=g) * 0.01
    d_h = (torch.randn(T, D, generator=g) * 0.01).bfloat16() if with_d_h else None
    return (dy if dy32 else dy.bfloat16()), h, w, rstd, d_h


def check_backward(dy, h, w, rstd, d_h, dx, dw):
    T, D = h.shape
    dx64, size, dw64, dw_size = rows64.norm_bwd(dy, h, w, rstd, d_h)
    bound = BF16_HALF_ULP * 1.001 * dx64.abs() + (chain(D) + 8) * U * size * 1.01 + 1e-40
    assert ((dx.double() - dx64).abs() <= bound).all()
    if dw is not None:
        assert ((dw.double() - dw64).abs() <= (T + 32) * U * dw_size + 1e-40).all()


@pytest.mark.parametrize("T,D", SHAPES + [(300, 2050), (700, 520), (1500, 96), (600, 4096), (1030, 5000), (300, 16640)])
def test_backward(T, D):
    for dy32, with_d_h in ((False, True), (True, False), (True, True)):
        print("backward", T, D, dy32, with_d_h, flush=True)
        args = bwd_inputs(T, D, dy32, with_d_h, seed=T + 3 * D)
        check_backward(*args, *run_backward(*args))


@pytest.mark.parametrize("D", [300, 4096, 20000])
def test_backward_in_place_and_without_dw(D):
    args = bwd_inputs(40, D, False, True, seed=5)
    dx, dw = run_backward(*args)
    assert torch.equal(run_backward(*args, inplace=True)[0], dx)
    assert torch.equal(run_backward(*args, want_dw=False)[0], dx)
    again = run_backward(*args)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)  # the same bits every time


def test_backward_of_no_rows_and_of_zero_rows():
    w = torch.ones(70, dtype=torch.bfloat16)
    dx, dw = run_backward(torch.zeros(0, 70), torch.zeros(0, 70).bfloat16(), w, torch.zeros(0), None)
    assert dx.shape == (0, 70) and (dw == 0).all()
    dy, h, w, _, _ = bwd_inputs(9, 70, False, False, seed=6)
    h[4] = 0
    rstd = (h.double().square().mean(1) + EPS).rsqrt().float()
    check_backward(dy, h, w, rstd, None, *run_backward(dy, h, w, rstd, None))


def test_backward_against_differences():
    # loss = sum(dy * y(h, w)) in 64 bits: central differences in h and w
    T, D = 6, 160
    dy, h, w, rstd, _ = bwd_inputs(T, D, True, False, seed=7)
    dx, dw = run_backward(dy, h, w, rstd, None)

    def loss(hh, ww):
        n = hh * (hh.square().mean(1, keepdim=True) + EPS) ** -0.5
        return (dy.double() * n * ww).sum()

    hd, wd = h.double(), w.double()
    scale = dx.double().abs().max()
    for t, d in [(0, 0), (1, 33), (3, 159), (5, 64), (2, 100)]:
        step = 1e-4 * float(hd[t].square().mean().sqrt())
        e = torch.zeros_like(hd)
        e[t, d] = step
        diff = (loss(hd + e, wd) - loss(hd - e, wd)) / (2 * step)
        # differences: order step^2; dx: half an ulp of bf16
        assert abs(float(dx[t, d]) - float(diff)) <= 2.0**-8 * abs(float(diff)) + 1e-5 * float(scale)
        e = torch.zeros_like(wd)
        e[d] = 1e-3
        diff = (loss(hd, wd + e) - loss(hd, wd - e)) / 2e-3
        assert abs(float(dw[d]) - float(diff)) <= 1e-5 * float(dw.abs().max())


def test_side_stream_and_graph():
    x, r, w = inputs(64, 1024, False, True, seed=8)
    want = run_forward(x, r, w, 128, False)
    dy, h, _, rstd, d_h = bwd_inputs(64, 1024, False, True, seed=9)
    want_dx, want_dw = run_backward(dy, h, w, rstd, d_h)
    xd, rd, wd = x.to(DEV), r.to(DEV), w.to(DEV)
    q, s = torch.empty_like(want[0], device=DEV), torch.empty_like(want[1], device=DEV)
    b = [t.to(DEV) for t in (dy, h, w, rstd)]
    dhd, dx, dw = d_h.to(DEV), torch.empty_like(want_dx, device=DEV), torch.empty_like(want_dw, device=DEV)
    ws = sq.rms_norm_bwd_workspace(64, 1024, DEV)

    def calls():
        sq.rms_norm_quant(xd, wd, q, s, residual=rd, eps=EPS)
        sq.rms_norm_bwd(*b, dx, dw=dw, d_h=dhd, workspace=ws)

    def check():
        torch.cuda.synchronize()
        assert torch.equal(q.cpu(), want[0]) and torch.equal(s.cpu(), want[1])
        assert torch.equal(dx.cpu(), want_dx) and torch.equal(dw.cpu(), want_dw)
        for t in (q, s, dx, dw):
            t.zero_()
        torch.cuda.synchronize()

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        calls()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(3):
        graph.replay()
        check()
        calls()
        check()
