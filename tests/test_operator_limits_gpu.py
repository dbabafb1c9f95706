"""The norm and microscaled operators past 2^32 elements, and at the ends of the
number range (GPU).  The last rows of a large call are compared with a small
call on those rows alone, bit for bit."""

import numpy as np
import pytest
import torch

import rows64
import swiglu_backward_int8_amd as sq

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    sq.lib()
    yield
    torch.cuda.empty_cache()


def new(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device=DEV)


def filled(R, K, seed=0):
    """bf16 [R, K] of cheap values: a few thousand random rows, repeated, each copy shifted by one column."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    base = torch.randn((4099, K), generator=g, device=DEV).bfloat16()
    x = new(R, K)
    for i in range(0, R, 4099):
        n = min(4099, R - i)
        x[i:i + n] = base[:n].roll(i // 4099, 1)
    return x


@pytest.mark.parametrize("D,group", [(4096, 128), (1000, 64)])
def test_norm_past_32_bits(D, group):
    T = 2**32 // D + 77
    x = filled(T, D)
    w = (1 + 0.1 * torch.randn(D, device=DEV)).bfloat16()

    def forward(x):
        T = x.shape[0]
        out = new(T, D, dtype=torch.int8), new(T, -(-D // group), dtype=torch.float32), new(T, dtype=torch.float32)
        sq.rms_norm_quant(x, w, out[0], out[1], rstd=out[2], group_size=group)
        return out

    tail = slice(T - 200, T)
    q, s, rstd = forward(x)
    small = forward(x[tail].clone())
    for a, b in zip((q, s, rstd), small):
        assert torch.equal(a[tail], b)
    v = new(T, D)
    sq.group_dequant(q, s, v, group_size=group)
    vs = new(200, D)
    sq.group_dequant(small[0], small[1], vs, group_size=group)
    assert torch.equal(v[tail], vs)
    del v
    # backward: rows are independent; dw of dy that is zero but in the last rows is theirs alone
    dy = torch.zeros_like(x)
    dy[tail] = filled(200, D, 1)
    dx, dw = new(T, D), new(D, dtype=torch.float32)
    sq.rms_norm_bwd(dy, x, w, rstd, dx, dw=dw, workspace=sq.rms_norm_bwd_workspace(T, D, DEV))
    dxs, dws = new(200, D), new(D, dtype=torch.float32)
    sq.rms_norm_bwd(dy[tail].clone(), x[tail].clone(), w, small[2], dxs, dw=dws,
                    workspace=sq.rms_norm_bwd_workspace(200, D, DEV))
    assert torch.equal(dx[tail], dxs)
    dx64, size, dw64, dw_size = rows64.norm_bwd(dy[tail].cpu(), x[tail].cpu(), w.cpu(), small[2].cpu())
    assert ((dw.cpu().double() - dw64).abs() <= 232 * 2.0**-24 * dw_size + 1e-40).all()


@pytest.mark.parametrize("K", [2048, 2001])
def test_mxfp4_past_32_bits(K):
    R = 2**32 // K + 100
    x = filled(R, K)
    sh = sq.mxfp4_shapes(R, K), sq.mxfp4_shapes(K, R)
    q, s, qt, st = (new(*t, dtype=torch.uint8) for pair in sh for t in pair)
    sq.mxfp4_quant(x, q, s, q_t=qt, s_t=st)
    first = (R // 32 - 3) * 32  # whole blocks of the columns from here on
    part = x[first:].clone()
    sh = sq.mxfp4_shapes(R - first, K), sq.mxfp4_shapes(K, R - first)
    small = [new(*t, dtype=torch.uint8) for pair in sh for t in pair]
    sq.mxfp4_quant(part, small[0], small[1], q_t=small[2], s_t=small[3])
    assert torch.equal(q[first:], small[0]) and torch.equal(s[first:], small[1])
    assert torch.equal(qt[:, first // 2:], small[2]) and torch.equal(st[:, first // 32:], small[3])
    only = torch.empty_like(q), torch.empty_like(s)
    sq.mxfp4_quant(x, *only)
    assert torch.equal(only[0], q) and torch.equal(only[1], s)
    v = new(R, K)
    sq.mxfp4_dequant(q, s, v)
    vs = new(R - first, K)
    sq.mxfp4_dequant(small[0], small[1], vs)
    assert torch.equal(v[first:], vs)


def codes(R, K, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.randint(0, 256, (R, K // 2), dtype=torch.uint8, device=DEV, generator=g)
    return q, torch.randint(126, 128, (R, K // 32), dtype=torch.uint8, device=DEV, generator=g)


def product(a, b, dtype=torch.float32):
    C = new(a[0].shape[0], b[0].shape[0], dtype=dtype)
    sq.mxfp4_gemm(*a, *b, C)
    return C


@pytest.mark.parametrize("M,N,K", [(70000, 62000, 64), (131200, 33000, 32), (2**32 // 32 + 50, 32, 128)])
def test_product_past_32_bits_of_results(M, N, K):
    a, b = codes(M, K, 1), codes(N, K, 2)
    C = product(a, b, torch.bfloat16)
    rows, cols = slice(M - 40, M), slice(max(0, N - 300), N)
    want = product([t[rows].clone() for t in a], [t[cols].clone() for t in b], torch.bfloat16)
    assert torch.equal(C[rows, cols], want)  # sums that fp32 holds exactly, whichever kernel adds them


@pytest.mark.parametrize("M,N", [(300000, 20), (12, 300000), (300000, 300)])
def test_product_past_32_bits_of_codes(M, N):
    K = 32768
    a, b = codes(M, K, 3), codes(N, K, 4)
    a[0].bitwise_and_(0x33), b[0].bitwise_and_(0x33)  # magnitudes up to 1.5: exact sums at this length
    C = product(a, b)
    rows, cols = slice(max(0, M - 30), M), slice(max(0, N - 30), N)
    va = rows64.mx_values(a[0][rows].cpu().numpy(), a[1][rows].cpu().numpy())
    vb = rows64.mx_values(b[0][cols].cpu().numpy(), b[1][cols].cpu().numpy())
    assert np.array_equal(C[rows, cols].cpu().double().numpy(), va @ vb.T)


@pytest.mark.parametrize("M,N", [(1, 16), (3, 40), (40, 40), (300, 300), (2000, 2100)])
def test_product_at_the_ends_of_the_exponents(M, N):
    # codes of 0.5: every sum is 2^(ea + eb - 254) * 64, down to fp32's subnormals and past its largest
    K = 256
    A, B = (torch.full((r, K // 2), 0x11, dtype=torch.uint8, device=DEV) for r in (M, N))
    for ea, eb in ((0, 127), (127, 0), (60, 64), (40, 80), (30, 82), (1, 110), (254, 121), (254, 122), (254, 254)):
        sA = torch.full((M, K // 32), ea, dtype=torch.uint8, device=DEV)
        sB = torch.full((N, K // 32), eb, dtype=torch.uint8, device=DEV)
        with np.errstate(over="ignore"):
            want = float(np.float32(2.0 ** (ea + eb - 254 + 6)) if ea + eb < 376 else np.float32(np.inf))
        assert (product((A, sA), (B, sB)) == want).all(), (ea, eb, want)
