"""The gated projection in bf16 and its backward pass (GPU).

Two kinds of inputs.  Small integers, whose sums fp32 holds exactly in any order:
gate and up (and dx and dw, with gates of 0 and 64, whose sigmoids are 1/2 and 1 in
fp32) have to be equal to the last bit.  And random ones, with u = 2^-24:
* a sum of K products is off by at most 2 K u of its terms' magnitudes S (K
  additions in some order, each a rounding of at most 2 u inside the matrix cores),
  and the rounding to bf16 adds at most 2^-8 of the value (half a step);
* y = silu(gate) * up: |silu'| <= 1.1, so 1.1 |up| times gate's error and |silu(gate)|
  times up's, and relative 4 (|gate| + 4) u for the sigmoid (the exponent's argument is
  rounded relative to itself, and the hardware's exp2 and division add a few u) and
  the two products;
* d_gu is within 4 (|gate| + 6) u of the magnitudes of its formula's terms, and half a
  step of bf16; dx and dw are compared with the products of the kernel's own d_gu.
"""

import pytest
import torch

import swiglu_backward_int8_amd as sq

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0**-24
HALF = 2.0**-8
bf16, f32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    sq.lib()


def new(*shape, dtype=bf16):
    return torch.full(shape, float("nan"), dtype=dtype, device=DEV)


def whole(T, H, D, seed):
    """Small whole numbers, few of them, so that sums of 2^20 of them stay below 2^24."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    pick = lambda *s: torch.randint(-3, 4, s, generator=g, device=DEV).to(bf16)
    return pick(T, D), pick(2 * H, D)


def normal(T, H, D, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((T, D), generator=g, device=DEV).to(bf16)
    w = (torch.randn((2 * H, D), generator=g, device=DEV) * max(D, 1) ** -0.5).to(bf16)
    return x, w


def silu(v):
    return v / (1 + torch.exp(-v))


def run_forward(x, w, gu=True):
    T, H = x.shape[0], w.shape[0] // 2
    y, kept = new(T, H), new(T, 2 * H) if gu else None
    sq.swiglu_gemm(x, w, y, gu=kept)
    torch.cuda.synchronize()
    return y, kept


def check_y(y, gate, up, e_gate, e_up):
    want = silu(gate) * up
    bound = HALF * 1.001 * want.abs() + 4 * (gate.abs() + 4) * U * want.abs() + 1.1 * up.abs() * e_gate + silu(gate).abs() * e_up
    assert ((y.double() - want).abs() <= bound + 1e-38).all()


# from single tokens to several tiles of every kind, rows and columns off all of them
SHAPES = [(1, 8, 8), (1, 64, 64), (1, 1024, 1000), (2, 72, 4096), (3, 8, 16), (5, 72, 40), (8, 264, 1376), (16, 128, 256), (17, 136, 200),
          (33, 512, 72), (40, 1000, 512), (64, 128, 256), (65, 200, 1024), (100, 2048, 128), (130, 264, 520), (200, 64, 2048), (256, 256, 64),
          (257, 520, 1032), (300, 1376, 264), (513, 72, 328), (777, 1376, 512), (1001, 1408, 1032), (2100, 1032, 136), (4, 11008, 4096),
          (31, 4096, 2048), (32, 136, 1000), (33, 72, 136), (47, 1376, 2048), (64, 4096, 264), (64, 4104, 128), (2050, 2056, 1096), (5000, 520, 264), (4097, 4104, 72)]


@pytest.mark.parametrize("T,H,D", SHAPES)
def test_forward(T, H, D):
    print("forward", T, H, D, flush=True)
    x, w = whole(T, H, D, T + H + D)
    y, gu = run_forward(x, w)
    want = x.double() @ w.double().t()
    assert torch.equal(gu, want.to(bf16))
    gate, up = want.chunk(2, 1)
    check_y(y, gate, up, 0.0, 0.0)
    assert torch.equal(run_forward(x, w, gu=False)[0], y)
    x, w = normal(T, H, D, T + H + D)
    y, gu = run_forward(x, w)
    want, size = x.double() @ w.double().t(), x.double().abs() @ w.double().abs().t()
    e = 2 * D * U * size
    assert ((gu.double() - want).abs() <= HALF * 1.001 * want.abs() + e).all()
    gate, up = want.chunk(2, 1)
    check_y(y, gate, up, *e.chunk(2, 1))


def run_backward(dy, gu, x, w, dx_dtype=bf16, dw_dtype=bf16, inplace=False, want=(True, True)):
    T, H, D = dy.shape[0], dy.shape[1], x.shape[1]
    gu = gu.clone()
    d_gu = gu if inplace else new(T, 2 * H)
    dx = new(T, D, dtype=dx_dtype) if want[0] else None
    dw = new(2 * H, D, dtype=dw_dtype) if want[1] else None
    ws = sq.swiglu_gemm_bwd_workspace(T, H, D, DEV).fill_(0xff)
    sq.swiglu_gemm_bwd(dy, gu, x, w, d_gu, dx=dx, dw=dw, workspace=ws)
    torch.cuda.synchronize()
    return d_gu, dx, dw


def check_d_gu(d_gu, dy, gu):
    gate, up = gu.double().chunk(2, 1)
    dy = dy.double()
    s = 1 / (1 + torch.exp(-gate))
    d_gate, d_up = dy * up * s * (1 + gate * (1 - s)), dy * gate * s
    size = (dy * up).abs() * s * (1 + gate.abs() * (1 - s))
    rel = 4 * (gate.abs() + 6) * U
    got = d_gu.double().chunk(2, 1)
    # 1 - s is off by s's error, relative to 1: gate times that
    assert ((got[0] - d_gate).abs() <= HALF * 1.001 * d_gate.abs() + rel * (size + (dy * up * gate).abs() * s) + 1e-38).all()
    assert ((got[1] - d_up).abs() <= HALF * 1.001 * d_up.abs() + rel * d_up.abs() + 1e-38).all()


def check_products(d_gu, x, w, dx, dw):
    d = d_gu.double()
    for got, a, b in ((dx, d, w.double()), (dw, d.t(), x.double())):
        if got is None:
            continue
        want, size = a @ b, a.abs() @ b.abs()
        half = HALF if got.dtype is bf16 else U
        assert ((got.double() - want).abs() <= half * 1.001 * want.abs() + 2 * a.shape[1] * U * size + 1e-38).all()


def whole_backward(T, H, D, seed):
    """dy, gu, x, w of whole numbers, gates 0 or 64: every d_gu is one too (or a half), and small."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    pick = lambda low, high, *s: torch.randint(low, high, s, generator=g, device=DEV).to(bf16)
    gate, up = 64 * pick(0, 2, T, H), pick(-1, 2, T, H)
    # a few gates of 64 alone, whose d_up is 64 dy
    gate = torch.where(torch.rand((T, H), generator=g, device=DEV) < 0.1, gate, torch.zeros_like(gate))
    return pick(-2, 3, T, H), torch.cat([gate, up], 1), pick(-2, 3, T, D), pick(-2, 3, 2 * H, D)


@pytest.mark.parametrize("T,H,D", SHAPES)
def test_backward(T, H, D):
    print("backward", T, H, D, flush=True)
    dy, gu, x, w = whole_backward(T, H, D, T + H + D)
    gate, up = gu.double().chunk(2, 1)
    s = torch.where(gate == 0, 0.5, 1.0)
    d = torch.cat([dy.double() * up * s, dy.double() * gate * s], 1)
    for dtype in (bf16, f32):
        d_gu, dx, dw = run_backward(dy, gu, x, w, dtype, dtype)
        assert torch.equal(d_gu, d.to(bf16))
        assert torch.equal(dx, (d @ w.double()).to(dtype))
        assert torch.equal(dw, (d.t() @ x.double()).to(dtype))
    x, w = normal(T, H, D, T + H + D)
    g = torch.Generator(device=DEV).manual_seed(T)
    gu = (torch.randn((T, 2 * H), generator=g, device=DEV) * 2).to(bf16)
    dy = (torch.randn((T, H), generator=g, device=DEV) * 0.01).to(bf16)
    out = run_backward(dy, gu, x, w)
    check_d_gu(out[0], dy, gu)
    check_products(out[0], x, w, *out[1:])
    again = run_backward(dy, gu, x, w, inplace=True)
    assert all(torch.equal(a, b) for a, b in zip(out, again))  # in place, and the same bits every time
    for want in ((True, False), (False, True), (False, False)):
        part = run_backward(dy, gu, x, w, want=want)
        assert all(b is None or torch.equal(a, b) for a, b in zip(out, part))


def test_no_rows_and_no_columns():
    x, w = normal(0, 16, 24, 0)
    y, gu = run_forward(x, w)
    assert y.shape == (0, 16) and gu.shape == (0, 32)
    d_gu, dx, dw = run_backward(new(0, 16), new(0, 32), x, w)
    assert dx.shape == (0, 24) and (dw == 0).all()
    x, w = normal(5, 0, 24, 0)
    assert run_forward(x, w)[0].shape == (5, 0)
    _, dx, dw = run_backward(new(5, 0), new(5, 0), x, w, f32, f32)
    assert (dx == 0).all() and dw.shape == (0, 24)
    x, w = normal(5, 16, 0, 0)
    y, gu = run_forward(x, w)
    assert (y == 0).all() and (gu == 0).all()
    dy, gu = torch.ones((5, 16), device=DEV).to(bf16), torch.ones((5, 32), device=DEV).to(bf16)
    check_d_gu(run_backward(dy, gu, x, w)[0], dy, gu)


@pytest.mark.parametrize("T,H,D", [(1, 64, 512), (40, 256, 256), (300, 264, 520), (1100, 1024, 320)])
def test_not_finite_values_stay_in_their_rows(T, H, D):
    x, w = normal(T, H, D, 1)
    y, gu = run_forward(x, w)
    t, h = T // 2, H // 3
    for bad in (float("inf"), float("nan")):
        xb, wb = x.clone(), w.clone()
        xb[t, D - 1] = bad
        got, got_gu = run_forward(xb, w)
        rest = torch.arange(T, device=DEV) != t
        assert torch.equal(got[rest], y[rest]) and torch.equal(got_gu[rest], gu[rest])
        assert not torch.isfinite(got_gu[t].float()).any()
        wb[h, 0] = bad
        got, got_gu = run_forward(x, wb)
        rest = torch.arange(H, device=DEV) != h
        assert torch.equal(got[:, rest], y[:, rest]) and torch.equal(got_gu[:, H:], gu[:, H:])
        assert not torch.isfinite(got_gu[:, h].float()).any()
    # backward: one bad gradient spoils its row of dx and its row of dw alone
    dy = (torch.randn((T, H), device=DEV) * 0.01).to(bf16)
    d_gu, dx, dw = run_backward(dy, gu, x, w)
    dyb = dy.clone()
    dyb[t, h] = float("nan")
    got = run_backward(dyb, gu, x, w)
    rest = torch.arange(T, device=DEV) != t
    assert torch.equal(got[1][rest], dx[rest]) and torch.isnan(got[1][t].float()).all()
    rest = torch.arange(2 * H, device=DEV) % H != h
    assert torch.equal(got[2][rest], dw[rest]) and torch.isnan(got[2][~rest].float()).all()


@pytest.mark.parametrize("T,H,D", [(1, 16, 16), (70, 128, 192), (260, 264, 136)])
def test_extreme_gates(T, H, D):
    # sums far past the exponential's range on both sides
    x = torch.full((T, D), 1.0, device=DEV).to(bf16)
    w = torch.zeros((2 * H, D), device=DEV)
    w[:H, 0] = torch.linspace(-400, 400, H, device=DEV)
    w[H:, 0] = 3.0
    w = w.to(bf16)
    y, gu = run_forward(x, w)
    gate, up = (x.double() @ w.double().t()).chunk(2, 1)
    check_y(y, gate, up, 0.0, 0.0)
    assert torch.isfinite(y.float()).all()
    dy = torch.ones((T, H), device=DEV).to(bf16)
    d_gu, dx, dw = run_backward(dy, gu, x, w)
    assert torch.isfinite(d_gu.float()).all()
    check_d_gu(d_gu, dy, gu)
    check_products(d_gu, x, w, dx, dw)


def formula(dy, gu):
    """d_gu in 64 bits."""
    gate, up = gu.double().chunk(2, 1)
    s = 1 / (1 + torch.exp(-gate))
    return torch.cat([dy.double() * up * s * (1 + gate * (1 - s)), dy.double() * gate * s], 1)


def test_d_gu_is_the_rounded_formula():
    # d_gu's fp32 values are off by 5e-9 of themselves on average before they are rounded, and so are another fp32 number in
    # at most 5e-9 / 2^-25 = 0.17 of the cases; that rounds to another bf16 number where one of the two is the middle between
    # two of them, 2 of 2^16, half of the times: 2.6e-6 of all.  (Rounding an fp32 computation: 1e-5.)
    T, H = 2048, 1024
    g = torch.Generator(device=DEV).manual_seed(5)
    gu = (torch.randn((T, 2 * H), generator=g, device=DEV) * 2).to(bf16)
    dy = torch.randn((T, H), generator=g, device=DEV).to(bf16)
    x, w = normal(T, H, 8, 0)
    d_gu = run_backward(dy, gu, x, w, want=(False, False))[0]
    assert (d_gu != formula(dy, gu).float().to(bf16)).sum() <= 2.6e-6 * d_gu.numel()


def test_d_gu_at_the_ends_of_the_range():
    # every combination: products past fp32's range that the sigmoid brings back, infinities, NaN, both zeros
    inf, nan = float("inf"), float("nan")
    values = torch.tensor([0.0, -0.0, 1.0, -1.0, 2.0**-126, 2.0**-133, -2.0**127, 2.0**127, 88.5, -88.5, 104.0, -104.0, -150.0, -700.0,
                           -800.0, -1000.0, 1000.0, 0.01, inf, -inf, nan, -1.28125, -1.2734375, -20.0], device=DEV)
    dy, gate, up = (v.reshape(-1) for v in torch.meshgrid(values, values, values, indexing="ij"))
    T = dy.numel()
    dy, gu = dy.to(bf16).reshape(T // 8, 8).contiguous(), torch.cat([gate.reshape(-1, 8), up.reshape(-1, 8)], 1).to(bf16)
    x, w = normal(T // 8, 8, 8, 0)
    d_gu = run_backward(dy, gu, x, w, want=(False, False))[0]
    gate, up = gu.double().chunk(2, 1)
    # in an order that no product of finite numbers leaves fp64's range in, and no small value is lost in
    e = torch.exp(-gate.abs())
    s, rest = torch.where(gate < 0, e, 1.0) / (1 + e), torch.where(gate < 0, 1.0, e) / (1 + e)
    want = torch.cat([dy.double() * up * (s * (1 + gate * rest)), dy.double() * (gate * s)], 1).float()
    got = d_gu.float()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.isnan(want).any() and torch.isinf(want).any()
    off = (got.double() - want.double()).abs()
    # half a step of bf16, 2^-134 among the denormal numbers, and what passes the largest one is infinite
    ok = torch.isnan(want) | (got == want) | (got == want.to(bf16).float()) | (off <= HALF * 1.001 * want.double().abs() + 2.0**-134 * 1.001)
    assert ok.all(), (got[~ok][:5], want[~ok][:5])


def test_gradients_against_differences():
    # loss = sum(dy * y(x, w)) in 64 bits, central differences in x and w; gate and up as they are (gu rounds them
    # by 2^-9 at most, which the gradients follow smoothly)
    T, H, D = 9, 40, 24
    x, w = normal(T, H, D, 5)
    dy = (torch.randn((T, H), generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)).to(bf16)
    _, gu = run_forward(x, w)
    _, dx, dw = run_backward(dy, gu, x, w, f32, f32)

    def loss(a, b):
        gate, up = (a @ b.t()).chunk(2, 1)
        return float((dy.double() * silu(gate) * up).sum())

    for got, which, places in ((dx, 0, [(0, 0), (3, 7), (8, 23), (5, 11)]), (dw, 1, [(0, 0), (39, 3), (40, 5), (79, 23), (17, 9)])):
        scale = float(got.abs().max())
        for at in places:
            hi, lo = [x.double(), w.double()], [x.double(), w.double()]
            hi[which], lo[which] = hi[which].clone(), lo[which].clone()
            hi[which][at] += 1e-4
            lo[which][at] -= 1e-4
            diff = (loss(*hi) - loss(*lo)) / 2e-4
            # gu and d_gu rounded: each term off by 2^-8 and by the rounded gate's and up's 2^-8 |gate|
            assert abs(float(got[at]) - diff) <= 4 * HALF * scale


@pytest.mark.parametrize("T,H,D", [(1, 1024, 512), (48, 512, 512), (520, 512, 264)])
def test_side_stream_and_graph(T, H, D):
    x, w = normal(T, H, D, 2)
    dy = (torch.randn((T, H), device=DEV) * 0.01).to(bf16)
    y, gu, d_gu, dx, dw = new(T, H), new(T, 2 * H), new(T, 2 * H), new(T, D), new(2 * H, D, dtype=f32)
    ws = sq.swiglu_gemm_bwd_workspace(T, H, D, DEV)
    outs = (y, gu, d_gu, dx, dw)

    def calls():
        sq.swiglu_gemm(x, w, y, gu=gu)
        sq.swiglu_gemm_bwd(dy, gu, x, w, d_gu, dx=dx, dw=dw, workspace=ws)

    def taken():
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        for t in outs:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        return got

    same = lambda a, b: all(torch.equal(u, v) for u, v in zip(a, b))
    calls()
    first = taken()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        calls()
    assert same(taken(), first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for i in range(4):
        if i == 2:
            x.copy_(normal(T, H, D, 9)[0])
            calls()
            first = taken()
        graph.replay()
        assert same(taken(), first)
        calls()
        assert same(taken(), first)
