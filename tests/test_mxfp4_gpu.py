"""Microscaled 4-bit codes, their product, and the dequantisers (GPU).

* Codes and exponents are exact: every bf16 value under every exponent a block
  can have, bit for bit.
* The product: with exponents in {126, 127} every partial sum is a whole number
  of quarters of the smallest product below 2^24 of them (36 * 4 * 4 * K for K
  <= 27000), so fp32 sums are exact in any order and C is compared for
  equality, which also shows any wrong, missing or doubled term.  With wide
  exponents each of the K additions rounds the running sum once: |error| <= K *
  2^-23 * sum |terms| (2^-23 allows for truncation inside the instruction).
* bf16 output adds half an ulp of bf16, 2^-8 of the magnitude.
"""

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


def quant(x, rows=True, cols=False):
    R, K = x.shape
    new = lambda shape: torch.full(shape, 0xAA, dtype=torch.uint8, device=DEV)
    q, s = map(new, sq.mxfp4_shapes(R, K)) if rows else (None, None)
    qt, st = map(new, sq.mxfp4_shapes(K, R)) if cols else (None, None)
    sq.mxfp4_quant(x.to(DEV), q, s, q_t=qt, s_t=st)
    torch.cuda.synchronize()
    return [None if t is None else t.cpu().numpy() for t in (q, s, qt, st)]


def check_quant(got, x):
    q, s, qt, st = got
    if q is not None:
        wq, ws = rows64.mx_quant(x)
        assert np.array_equal(s, ws) and np.array_equal(q, wq)
    if qt is not None:
        wq, ws = rows64.mx_quant(x.t())
        assert np.array_equal(st, ws) and np.array_equal(qt, wq)


def every_bf16():
    """Blocks of 32 that hold every finite bf16 value below, at and just above each power of two:
    per exponent, a leading value that sets it and 31 others of the same or smaller exponents."""
    bits = torch.arange(0x7F80, dtype=torch.int32)
    rows = []
    for e in range(0, 255):
        lead = (e << 7) | 0x40
        mine = bits[(bits >> 7 <= e) & (bits >> 7 >= e - 5)]
        mine = torch.cat([mine, mine | 0x8000])
        mine = torch.cat([mine, torch.zeros(-len(mine) % 31, dtype=torch.int32)]).view(-1, 31)
        rows.append(torch.cat([torch.full((mine.shape[0], 1), lead, dtype=torch.int32), mine], 1))
    b = torch.cat(rows).to(torch.int32)
    b = torch.where(b >= 0x8000, b - 0x10000, b).to(torch.int16)
    return b.view(torch.bfloat16)


def test_quant_every_value_and_exponent():
    x = every_bf16()
    check_quant(quant(x), x)
    xt = x.t().contiguous()  # [32, n]: blocks along the columns
    check_quant(quant(xt, rows=False, cols=True), xt)


def test_dequant_every_code_and_exponent():
    s = torch.arange(256, dtype=torch.uint8).repeat_interleave(8).view(256, 8)
    q = torch.arange(256, dtype=torch.uint8).repeat(128).view(256, 128)
    out = torch.empty((256, 256), dtype=torch.bfloat16, device=DEV)
    sq.mxfp4_dequant(q.to(DEV), s.to(DEV), out)
    want = torch.from_numpy(rows64.mx_values(q.numpy(), s.numpy()).astype(np.float32)).bfloat16()
    got = out.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    fine = ~torch.isnan(want)
    assert torch.equal(got[fine].view(torch.int16), want[fine].view(torch.int16))


SHAPES = [(1, 1), (1, 31), (1, 32), (1, 33), (3, 7), (32, 32), (33, 31), (31, 64), (64, 511), (65, 512), (100, 513),
          (1, 11008), (7, 4096), (256, 1376), (129, 1001), (200, 2050), (1030, 96), (2, 22016), (513, 520)]


def values(R, K, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, K, generator=g) * torch.exp2(torch.randint(-20, 20, (R, K), generator=g) / 4.0)
    x[::5, ::3] = 0
    if R > 3:
        x[3] = 0
    return x.bfloat16()


@pytest.mark.parametrize("R,K", SHAPES)
def test_quant_and_dequant(R, K):
    x = values(R, K, R + K)
    rows = quant(x)
    both = quant(x, cols=True)
    cols = quant(x, rows=False, cols=True)
    check_quant(rows, x)
    check_quant(both, x)
    check_quant(cols, x)
    out = torch.full((R, K), float("nan"), dtype=torch.bfloat16, device=DEV)
    sq.mxfp4_dequant(torch.from_numpy(rows[0]).to(DEV), torch.from_numpy(rows[1]).to(DEV), out)
    want = rows64.mx_values(rows[0], rows[1])[:, :K]
    assert np.array_equal(out.cpu().double().numpy(), want)


def test_quant_of_many_blocks():
    x = values(4500, 1120, 3)  # more than one round of the walk per workgroup
    check_quant(quant(x), x)
    x = values(4500, 1001, 4)
    check_quant(quant(x), x)
    for R, K in ((8200, 2048), (8192, 2048), (8195, 2050), (40000, 100), (40001, 5)):  # the wider bands
        x = values(R, K, R + K)
        check_quant(quant(x, cols=True), x)


@pytest.mark.parametrize("R,K", [
    (1, 1), (1, 9), (2, 10), (31, 9), (33, 11), (127, 129), (128, 129), (129, 127), (129, 136), (256, 264), (257, 250),
    (255, 393), (160, 135), (161, 512), (300, 8), (300, 7),
    (3329, 3849), (3329, 3848), (3328, 3855), (3297, 3842), (49153, 9), (49153, 5), (6400, 2049), (6401, 2048)])
def test_quant_of_both_axes_at_the_edges(R, K):
    # tiles that reach past the rows, the columns or both, in tensors of both
    # tile sizes; what lies around x is NaN and would show in the exponents
    print("quant", R, K, flush=True)
    x = values(R, K, R + K)
    room = torch.full((R * K + 1040,), float("nan"), dtype=torch.bfloat16, device=DEV)
    inside = room[520:520 + R * K].view(R, K)
    inside.copy_(x)
    for rows in (True, False):
        check_quant(quant(inside, rows=rows, cols=True), x)


def test_quant_blocks_that_are_not_finite():
    x = values(40, 200, 5)
    x[1, 40], x[2, 199], x[3, 0], x[39, 64] = float("inf"), float("nan"), -float("inf"), float("nan")
    q, s, qt, st = quant(x, cols=True)
    for got_q, got_s, y in ((q, s, x), (qt, st, x.t())):
        wq, ws = rows64.mx_quant(y)
        assert np.array_equal(got_s, ws) and (ws == 255).sum() == 4
        fine = np.repeat(ws != 255, 16, 1)
        assert np.array_equal(got_q[fine], wq[fine])
    out = torch.empty((40, 200), dtype=torch.bfloat16, device=DEV)
    sq.mxfp4_dequant(torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV), out)
    assert np.array_equal(np.isnan(out.cpu().float().numpy()), np.repeat(s == 255, 32, 1)[:, :200])


@pytest.mark.parametrize("R,K", [(1, 1), (3, 7), (5, 33), (64, 128), (100, 1001), (2, 22016), (300, 520), (4200, 1100)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_group_dequant(R, K, group):
    rng = np.random.default_rng(R + K + group)
    s = (rng.random((R, -(-K // group))) * 10.0 ** rng.integers(-6, 3, (R, 1))).astype(np.float32)
    wide = np.repeat(s, group, 1)[:, :K]
    q8 = rng.integers(-127, 128, (R, K)).astype(np.int8)
    fp = rng.integers(0, 256, (R, K)).astype(np.uint8)
    fp[(fp & 127) == 127] = 0  # the NaN patterns
    for q, v in ((torch.from_numpy(q8), q8.astype(np.float32)),
                 (torch.from_numpy(fp), torch.from_numpy(fp).view(torch.float8_e4m3fn).float().numpy())):
        out = torch.full((R, K), float("nan"), dtype=torch.bfloat16, device=DEV)
        sq.group_dequant(q.to(DEV), torch.from_numpy(s).to(DEV), out, group_size=group)
        want = torch.from_numpy(v * wide).bfloat16()
        got = out.cpu()
        assert torch.equal(got.float(), want.float())


# ---- the product ----

def operands(M, N, K, exponents, seed):
    rng = np.random.default_rng(seed)
    make = lambda R: (rng.integers(0, 256, (R, K // 2)).astype(np.uint8),
                      rng.integers(exponents[0], exponents[1] + 1, (R, K // 32)).astype(np.uint8))
    return make(M) + make(N)


def run_gemm(A, sA, B, sB, out=torch.float32):
    C = torch.full((A.shape[0], B.shape[0]), float("nan"), dtype=out, device=DEV)
    sq.mxfp4_gemm(*(torch.from_numpy(t).to(DEV) for t in (A, sA, B, sB)), C)
    torch.cuda.synchronize()
    return C.cpu()


GEMM_SHAPES = [(1, 1, 32), (1, 16, 32), (1, 17, 64), (1, 4096, 4096), (1, 1000, 11008), (2, 50, 96), (5, 33, 480),
               (8, 2048, 512), (15, 100, 544), (16, 16, 512), (16, 1024, 1376), (17, 40, 1024), (31, 63, 160),
               (33, 130, 2048), (48, 512, 2080), (64, 4096, 1024), (65, 65, 65 * 32), (100, 300, 256), (127, 129, 352),
               (128, 128, 128), (128, 1024, 4096), (200, 250, 288), (255, 257, 256), (256, 256, 512), (256, 512, 768),
               (300, 1001, 1376), (513, 511, 1056), (512, 768, 224), (777, 1001, 1376), (1024, 1024, 1024),
               (1030, 2060, 544), (4400, 4352, 128), (4352, 4400, 1152), (4360, 4352, 2144), (5000, 4096, 32), (200, 129, 32), (33, 1024, 4096),
               (60, 2000, 896), (64, 4096, 1408), (120, 4000, 1152), (250, 4000, 640), (20, 9000, 256), (300, 3, 32), (5000, 2, 64),
               (1400, 2000, 128), (1408, 2048, 384), (1400, 2001, 896), (1401, 2000, 1152), (1290, 1290, 2176),
               (2176, 2200, 640), (2048, 300, 96), (3000, 17, 640), (9, 3000, 32), (1500, 2100, 2048)]


@pytest.mark.parametrize("M,N,K", GEMM_SHAPES)
def test_product_is_exact_where_fp32_is(M, N, K):
    print("product", M, N, K, flush=True)
    ops = operands(M, N, K, (126, 127), M + N + K)
    want = rows64.mx_values(*ops[:2]) @ rows64.mx_values(*ops[2:]).T
    got = run_gemm(*ops)
    assert np.array_equal(got.double().numpy(), want)
    # bf16: the same sums, rounded once
    got = run_gemm(*ops, out=torch.bfloat16)
    assert torch.equal(got, torch.from_numpy(want.astype(np.float32)).bfloat16())


@pytest.mark.parametrize("M,N,K", [(4352, 4353, 160), (4300, 4370, 1152), (1536, 1540, 256), (1664, 1665, 96)])
def test_product_of_whole_tiles_in_rows_off_the_lines(M, N, K):
    test_product_is_exact_where_fp32_is(M, N, K)


@pytest.mark.parametrize("M,N,K", [(1, 500, 4096), (40, 70, 11008), (129, 260, 2048), (600, 700, 1376)])
def test_product_of_wide_exponents(M, N, K):
    ops = operands(M, N, K, (107, 147), 9)
    a, b = rows64.mx_values(*ops[:2]), rows64.mx_values(*ops[2:])
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    got = run_gemm(*ops).double().numpy()
    assert (np.abs(got - want) <= K * 2.0**-23 * size).all()
    bound = K * 2.0**-23 * size
    got = run_gemm(*ops, out=torch.bfloat16).double().numpy()
    assert (np.abs(got - want) <= bound + 2.0**-8 * 1.001 * (np.abs(want) + bound)).all()


@pytest.mark.parametrize("M,N,K", [(1, 40, 512), (70, 90, 544), (300, 300, 1024)])
def test_product_of_nan_exponents(M, N, K):
    A, sA, B, sB = operands(M, N, K, (126, 127), 10)
    sA[M // 2, 3] = 255
    sB[7, K // 32 - 1] = 255
    got = run_gemm(A, sA, B, sB)
    bad = np.zeros((M, N), bool)
    bad[M // 2] = True
    bad[:, 7] = True
    assert np.array_equal(np.isnan(got.numpy()), bad)


@pytest.mark.parametrize("M,N", [(1, 8), (50, 60), (300, 257)])
def test_product_over_no_values_is_zero(M, N):
    e = np.zeros((M, 0), np.uint8), np.zeros((N, 0), np.uint8)
    assert (run_gemm(e[0], e[0], e[1], e[1]) == 0).all()


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_product_of_unaligned_exponents_and_into_an_unaligned_result(out):
    # C only has to be aligned to its elements
    # and exponents to nothing: K of whole words of them, from odd addresses
    for shape in ((20, 36, 320), (200, 310, 320), (40, 300, 1024), (1500, 1400, 384)):
        ops = operands(*shape, (126, 127), 12)
        M, N = shape[:2]
        want = torch.from_numpy((rows64.mx_values(*ops[:2]) @ rows64.mx_values(*ops[2:]).T).astype(np.float32))
        buf = torch.full((M * N + 2,), 7.0, dtype=out, device=DEV)
        A, sA, B, sB = (torch.from_numpy(t).to(DEV) for t in ops)
        odd = lambda t: torch.cat([t.new_full((3,), 255), t.flatten()])[3:].view(t.shape)
        sq.mxfp4_gemm(A, odd(sA), B, odd(sB), buf[1:1 + M * N].view(M, N))
        got = buf.cpu()
        assert torch.equal(got[1:-1].view(M, N), want.to(out)) and got[0] == 7 and got[-1] == 7


def test_training_step_through_both_axes():
    # y = x w^T: forward and both gradients contract over different axes; each
    # product is compared with the 64-bit product of its own operands' values
    T, H, D = 96, 160, 224
    x, w, dy = values(T, D, 20), values(H, D, 21), values(T, H, 22)
    d = lambda t: t.to(DEV)
    q = {n: [None if t is None else torch.from_numpy(t).to(DEV) for t in quant(t0, cols=True)]
         for n, t0 in (("x", x), ("w", w), ("dy", dy))}
    for a, sa, b, sb, shape in ((*q["x"][:2], *q["w"][:2], (T, H)),       # y = x . w^T
                                (*q["dy"][:2], *q["w"][2:], (T, D)),      # dx = dy . w
                                (*q["dy"][2:], *q["x"][2:], (H, D))):     # dw = dy^T . x
        C = torch.empty(shape, device=DEV)
        sq.mxfp4_gemm(a, sa, b, sb, C)
        va, vb = (rows64.mx_values(u.cpu().numpy(), v.cpu().numpy()) for u, v in ((a, sa), (b, sb)))
        want, size = va @ vb.T, np.abs(va) @ np.abs(vb).T
        assert (np.abs(C.cpu().double().numpy() - want) <= va.shape[1] * 2.0**-23 * size).all()


def test_side_stream_and_graph():
    x = values(130, 1024, 30)
    want = quant(x, cols=True)
    wq, ws, _, _ = (torch.from_numpy(t).to(DEV) if t is not None else None for t in quant(values(512, 1024, 31)))
    xd = x.to(DEV)
    q, s, qt, st = (torch.empty(t.shape, dtype=torch.uint8, device=DEV) for t in want)
    C, one = torch.empty((130, 512), device=DEV), torch.empty((1, 512), device=DEV)
    out = torch.empty_like(xd)

    def calls():
        sq.mxfp4_quant(xd, q, s, q_t=qt, s_t=st)
        sq.mxfp4_gemm(q, s, wq, ws, C)
        sq.mxfp4_gemm(q[:1], s[:1], wq, ws, one)
        sq.mxfp4_dequant(q, s, out)

    calls()
    torch.cuda.synchronize()
    first = [t.clone() for t in (q, s, qt, st, C, one, out)]
    assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(first, want))

    def check():
        torch.cuda.synchronize()
        for a, b in zip((q, s, qt, st, C, one, out), first):
            assert torch.equal(a, b)
            a.zero_()
        torch.cuda.synchronize()

    check()
    with torch.cuda.stream(torch.cuda.Stream()):
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
