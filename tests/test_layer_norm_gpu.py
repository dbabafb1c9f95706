"""The layer norm with its dropout and quantised output, its backward pass, and the
dropout alone (GPU).

Bounds, with u = 2^-24, a row's longest chain of additions L = 8 ceil(D / 512) + 32
(a lane's elements, then the joins), and A the mean magnitude of a row:
* the mask is the generator's, bit for bit; h (and dropout_add's output) is one
  fp32 product and one fp32 sum rounded to bf16: equal bits.
* mean: (L + 2) u A.
* rstd: each difference from the mean is off by the mean's error and a rounding,
  whose square adds at most the mean's error squared (the differences' sum is zero)
  and relative errors; a wave's own mean stands in for the row's, and the joins
  give the same sum.  With s the standard deviation and e = (L + 2) u A: relative
  (L / 2 + 8) u + (e / s)^2 + u A / s, where eps only makes it smaller.
* y before rounding: the mean's error and rstd's, four roundings, and the rounding to
  bf16 adds at most 2^-8 of its magnitude (half a unit in the last place).
* codes and scales are those of the kernel's own y_bf16, bit for bit.
* dx: 2 L + 12 roundings of the magnitudes it is made of, and half an ulp of bf16;
  dx_drop the same numbers times the scale.
* dw, db: T + 32 roundings of the sums of their terms' magnitudes (dw two more in n).
"""

import numpy as np
import pytest
import torch

import ln64
import rows64
import swiglu_backward_int8_amd as sq

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0**-24
BF16_HALF_ULP = 2.0**-8
EPS = 1e-5
RNG = (0x123456789ABCDEF, -987654321)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    sq.lib()


def rng_tensor(rng=RNG):
    return torch.tensor(rng, dtype=torch.int64, device=DEV)


def inputs(T, D, x32, residual, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, D, generator=g) * torch.exp(torch.randn(T, 1, generator=g)) + torch.randn(T, 1, generator=g)
    x[:, ::37] *= 30.0
    x[5::11] = 0
    r = torch.randn(T, D, generator=g).bfloat16() if residual else None
    if residual:
        r[5::11] = 0
    w = (1 + 0.3 * torch.randn(D, generator=g)).bfloat16()
    b = (0.2 * torch.randn(D, generator=g)).bfloat16()
    return (x if x32 else x.bfloat16()), r, w, b


def chain(D):
    return 8 * -(-D // 512) + 32


def run_forward(x, r, w, b, group, e4m3, y_q=True, y_bf16=True, eps=EPS, inplace=False, p=0.0, offset=0):
    T, D = x.shape
    q = torch.full((T, D), 55, dtype=torch.uint8 if e4m3 else torch.int8, device=DEV) if y_q else None
    s = torch.full((T, -(-D // group)), float("nan"), device=DEV) if y_q else None
    y = torch.full((T, D), float("nan"), dtype=torch.bfloat16, device=DEV) if y_bf16 else None
    rd = None if r is None else r.to(DEV)
    h = rd if inplace else torch.full((T, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    mean, rstd = (torch.full((T,), float("nan"), device=DEV) for _ in range(2))
    sq.layer_norm_quant(x.to(DEV), w.to(DEV), bias=None if b is None else b.to(DEV), y_q=q, y_s=s, residual=rd, h=h, mean=mean,
                        rstd=rstd, y_bf16=y, eps=eps, group_size=group, p=p, rng=rng_tensor() if p > 0 else None, offset=offset)
    torch.cuda.synchronize()
    return [None if t is None else t.cpu() for t in (q, s, y, h, mean, rstd)]


def check_forward(x, r, w, b, out, group, e4m3, eps=EPS, p=0.0, offset=0):
    q, s, y, h, mean, rstd = out
    D = x.shape[1]
    want_h = ln64.stream(x, r, p, RNG, offset)
    assert torch.equal(h.view(torch.int16), want_h.view(torch.int16))
    mean64, rstd64, y64, size = ln64.norm(want_h, w, b, eps)
    A = want_h.double().abs().mean(1)
    e = (chain(D) + 2) * U * A
    assert ((mean.double() - mean64).abs() <= e + 1e-40).all()
    rel = (chain(D) / 2 + 8) * U + (e * rstd64) ** 2 + U * A * rstd64
    assert ((rstd.double() - rstd64).abs() <= rel * rstd64).all()
    if y is not None:
        bound = BF16_HALF_ULP * 1.001 * y64.abs() + (rel[:, None] + 4 * U) * size
        bound += ((e + U * A) * rstd64)[:, None] * w.double().abs() + 1e-40
        assert ((y.double() - y64).abs() <= bound).all()
    if q is not None and y is not None:
        codes, scales = rows64.group_quant(y, group, e4m3)
        assert np.array_equal(q.view(torch.uint8).numpy(), codes)
        assert np.array_equal(s.numpy(), scales)


SHAPES = [(1, 1), (1, 4096), (3, 7), (2, 31), (5, 32), (4, 33), (7, 128), (9, 200), (6, 511), (6, 512), (5, 513),
          (33, 1001), (20, 1024), (3, 1025), (3, 1376), (4, 2048), (3, 2050), (5, 4095), (2, 4096), (3, 4097), (2, 8192), (3, 8200),
          (2, 11008), (2, 12289), (1, 16384), (2, 16385), (2, 22016), (1, 70001)]


@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("group,e4m3,p", [(128, False, 0.0), (64, True, 0.1), (32, False, 0.5), (32, True, 0.0)])
def test_forward(T, D, group, e4m3, p):
    x, r, w, b = inputs(T, D, x32=(T + D) % 2 == 1, residual=D % 3 != 0, seed=T * 7 + D)
    if D % 5 == 0:
        b = None
    print("forward", T, D, group, e4m3, p, flush=True)
    check_forward(x, r, w, b, run_forward(x, r, w, b, group, e4m3, p=p, offset=D), group, e4m3, p=p, offset=D)


@pytest.mark.parametrize("T,D", [(2500, 1376), (2304, 4096), (2060, 1001), (4097, 512), (2049, 96), (2111, 2048)])
def test_forward_many_rows(T, D):
    for x32, e4m3, p in ((False, False, 0.0), (True, True, 0.2)):
        print("forward", T, D, x32, e4m3, p, flush=True)
        x, r, w, b = inputs(T, D, x32, True, seed=D)
        check_forward(x, r, w, b, run_forward(x, r, w, b, 128, e4m3, p=p), 128, e4m3, p=p)


@pytest.mark.parametrize("D", [64, 1000, 4096, 20000])
def test_forward_of_rows_far_from_zero(D):
    # an offset of 100 standard deviations, each row another: the squares are those of the differences
    g = torch.Generator().manual_seed(D)
    x = torch.randn(6, D, generator=g) + 100 * torch.randn(6, 1, generator=g)
    w, b = (1 + 0.3 * torch.randn(D, generator=g)).bfloat16(), torch.randn(D, generator=g).bfloat16()
    check_forward(x, None, w, b, run_forward(x, None, w, b, 128, False), 128, False)


@pytest.mark.parametrize("D", [257, 4096, 20000])
def test_forward_in_place_and_optional_outputs(D):
    x, r, w, b = inputs(4, D, False, True, seed=1)
    for p in (0.0, 0.3):
        full = run_forward(x, r, w, b, 64, False, p=p)
        inplace = run_forward(x, r, w, b, 64, False, inplace=True, p=p)
        for a, c in zip(full, inplace):
            assert torch.equal(a, c)
        only_y = run_forward(x, r, w, b, 64, False, y_q=False, p=p)
        only_q = run_forward(x, r, w, b, 64, False, y_bf16=False, p=p)
        assert torch.equal(only_y[2], full[2]) and torch.equal(only_q[0], full[0]) and torch.equal(only_q[1], full[1])
        # without h and statistics: the wide rows make h again
        q, s = torch.empty_like(full[0], device=DEV), torch.empty_like(full[1], device=DEV)
        sq.layer_norm_quant(x.to(DEV), w.to(DEV), b.to(DEV), q, s, residual=r.to(DEV), eps=EPS, group_size=64, p=p,
                            rng=rng_tensor() if p > 0 else None)
        assert torch.equal(q.cpu(), full[0]) and torch.equal(s.cpu(), full[1])


@pytest.mark.parametrize("D", [40, 640, 4096, 17000])
def test_not_finite_rows(D):
    # an infinity or a NaN makes its row NaN, and shows in the scales there; a dropped one is 0
    x, r, w, b = inputs(5, D, False, True, seed=4)
    want = run_forward(x, r, w, b, 128, False)
    for bad in (float("inf"), float("nan")):
        y = x.clone()
        y[2, 30] = bad
        got = run_forward(y, r, w, b, 128, False)
        for a, c in zip(got, want):
            assert torch.equal(a[[0, 1, 3, 4]], c[[0, 1, 3, 4]])
        assert torch.isnan(got[1][2]).all() and torch.isnan(got[2][2]).all()
    p = 0.5
    keep = ln64.kept(RNG, 5, D, p)
    x = torch.where(keep, x, torch.tensor(float("nan")).bfloat16())
    check_forward(torch.where(keep, x, torch.zeros(()).bfloat16()), r, w, b, run_forward(x, r, w, b, 128, False, p=p), 128, False, p=p)


def test_rows_of_one_value():
    # variance zero up to the mean's rounding: y is the bias, up to that over sqrt(eps)
    for D in (7, 512, 1000, 4096, 20000):
        x = torch.tensor([0.0, 1.0, -3.140625, 1000.0])[:, None].expand(4, D).contiguous().bfloat16()
        w, b = torch.ones(D).bfloat16(), torch.linspace(-1, 1, D).bfloat16()
        check_forward(x, None, w, b, run_forward(x, None, w, b, 128, False), 128, False)


def run_backward(dy, h, w, mean, rstd, d_h, sums=(True, True), inplace=False, p=0.0, offset=0):
    T, D = h.shape
    dd = None if d_h is None else d_h.to(DEV)
    dx = dd if inplace else torch.full((T, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    drop = torch.full((T, D), float("nan"), dtype=torch.bfloat16, device=DEV) if p > 0 else None
    dw, db = (torch.full((D,), float("nan"), device=DEV) if want else None for want in sums)
    ws = sq.layer_norm_bwd_workspace(T, D, DEV).fill_(0xff) if any(sums) or D > 16384 else None
    sq.layer_norm_bwd(dy.to(DEV), h.to(DEV), w.to(DEV), mean.to(DEV), rstd.to(DEV), dx, dw=dw, db=db, d_h=dd, dx_drop=drop,
                      workspace=ws, p=p, rng=rng_tensor() if p > 0 else None, offset=offset)
    torch.cuda.synchronize()
    return [None if t is None else t.cpu() for t in (dx, drop, dw, db)]


def bwd_inputs(T, D, dy32, with_d_h, seed):
    g = torch.Generator().manual_seed(seed)
    h = (torch.randn(T, D, generator=g) * torch.exp(torch.randn(T, 1, generator=g)) + torch.randn(T, 1, generator=g)).bfloat16()
    w = (1 + 0.3 * torch.randn(D, generator=g)).bfloat16()
    mean = h.double().mean(1)
    rstd = ((h.double() - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
    dy = torch.randn(T, D, generator=g) * 0.01
    d_h = (torch.randn(T, D, generator=g) * 0.01).bfloat16() if with_d_h else None
    return (dy if dy32 else dy.bfloat16()), h, w, mean.float(), rstd, d_h


def check_backward(dy, h, w, mean, rstd, d_h, out, p=0.0, offset=0):
    dx, drop, dw, db = out
    T, D = h.shape
    dx64, size, dw64, dw_size, db64, db_size = ln64.norm_bwd(dy, h, w, mean, rstd, d_h)
    err = (2 * chain(D) + 12) * U * size * 1.01 + 1e-40
    assert ((dx.double() - dx64).abs() <= BF16_HALF_ULP * 1.001 * dx64.abs() + err).all()
    if drop is not None:
        k = ln64.kept(RNG, T, D, p, offset)
        s = ln64.scale(p)
        assert (drop[~k] == 0).all()
        bound = s * (BF16_HALF_ULP * 1.001 * dx64.abs() + err + U * dx64.abs())
        assert ((drop.double() - dx64 * s).abs()[k] <= bound[k]).all()
    if dw is not None:
        assert ((dw.double() - dw64).abs() <= (T + 34) * U * dw_size + 1e-40).all()
    if db is not None:
        assert ((db.double() - db64).abs() <= (T + 32) * U * db_size + 1e-40).all()


@pytest.mark.parametrize("T,D", SHAPES + [(300, 2050), (700, 520), (1500, 96), (600, 4096), (1030, 5000), (300, 16640), (270, 9001)])
def test_backward(T, D):
    for dy32, with_d_h, p in ((False, True, 0.0), (True, False, 0.1), (False, False, 0.6), (True, True, 0.0)):
        print("backward", T, D, dy32, with_d_h, p, flush=True)
        args = bwd_inputs(T, D, dy32, with_d_h, seed=T + 3 * D)
        check_backward(*args, run_backward(*args, p=p, offset=3), p=p, offset=3)


@pytest.mark.parametrize("D", [300, 4096, 10000, 20000])
def test_backward_in_place_and_without_sums(D):
    args = bwd_inputs(40, D, False, True, seed=5)
    full = run_backward(*args, p=0.1)
    same = lambda a, b: all(u is None or v is None or torch.equal(u, v) for u, v in zip(a, b))
    assert same(run_backward(*args, inplace=True, p=0.1), full)
    for sums in ((False, False), (True, False), (False, True)):
        assert same(run_backward(*args, sums=sums, p=0.1), full)
    assert torch.equal(run_backward(*args)[0], full[0])
    assert same(run_backward(*args, p=0.1), full)  # the same bits every time


def test_backward_of_no_rows():
    w = torch.ones(70, dtype=torch.bfloat16)
    none = torch.zeros(0)
    dx, _, dw, db = run_backward(torch.zeros(0, 70), torch.zeros(0, 70).bfloat16(), w, none, none, None)
    assert dx.shape == (0, 70) and (dw == 0).all() and (db == 0).all()


def test_backward_against_differences():
    # loss = sum(dy * y(x, w, b)) with y's dropout, in 64 bits: central differences in x, w and b
    T, D, p = 6, 160, 0.25
    g = torch.Generator().manual_seed(7)
    x = torch.randn(T, D, generator=g).bfloat16()
    r = (torch.randn(T, D, generator=g) + 0.5).bfloat16()
    w = (1 + 0.3 * torch.randn(D, generator=g)).bfloat16()
    b = torch.randn(D, generator=g).bfloat16()
    dy = torch.randn(T, D, generator=g) * 0.01
    _, _, _, h, mean, rstd = run_forward(x, r, w, b, 128, False, p=p)
    dx, drop, dw, db = run_backward(dy, h, w, mean, rstd, None, p=p)
    k, s = ln64.kept(RNG, T, D, p), ln64.scale(p)
    # the rounding of h is no part of the function: the differences start from the rounded h
    rest = h.double() - torch.where(k, x.double() * s, 0.0)

    def loss(xx, rr, ww, bb):
        hh = rr + torch.where(k, xx * s, 0.0)
        d = hh - hh.mean(1, keepdim=True)
        n = d * (d.square().mean(1, keepdim=True) + EPS) ** -0.5
        return float((dy.double() * (n * ww + bb)).sum())

    base = [x.double(), rest, w.double(), b.double()]
    for got, which in ((drop, 0), (dx, 1)):
        scale = float(got.double().abs().max())
        for t, d in [(0, 0), (1, 33), (3, 159), (5, 64), (2, 100), (4, 7)]:
            hi, lo = [v.clone() for v in base], [v.clone() for v in base]
            hi[which][t, d] += 1e-4
            lo[which][t, d] -= 1e-4
            diff = (loss(*hi) - loss(*lo)) / 2e-4
            assert abs(float(got[t, d]) - diff) <= 2.0**-8 * abs(diff) + 1e-5 * scale
    for got, which in ((dw, 2), (db, 3)):
        for d in (0, 33, 100, 159):
            hi, lo = [v.clone() for v in base], [v.clone() for v in base]
            hi[which][d] += 1e-3
            lo[which][d] -= 1e-3
            assert abs(float(got[d]) - (loss(*hi) - loss(*lo)) / 2e-3) <= 1e-5 * float(got.abs().max())


@pytest.mark.parametrize("T,D", SHAPES + [(700, 96), (300, 1000), (64, 4096), (33, 11008)])
@pytest.mark.parametrize("x32", [False, True])
def test_dropout(T, D, x32):
    x, r, _, _ = inputs(T, D, x32, True, seed=T + D)
    xd, rd, rng = x.to(DEV), r.to(DEV), rng_tensor()
    bits = lambda t: t.cpu().view(torch.int16)
    for p, res, offset in ((0.1, True, 0), (0.5, False, 2**40), (0.0, True, 0), (0.999, False, -1)):
        print("dropout", T, D, x32, p, res, flush=True)
        out = torch.full((T, D), float("nan"), dtype=torch.bfloat16, device=DEV)
        sq.dropout_add(xd, out, p, rng, residual=rd if res else None, offset=offset)
        want = ln64.stream(x, r if res else None, p, RNG, offset)
        assert torch.equal(bits(out), bits(want))
    place = rd.clone()
    sq.dropout_add(xd, place, 0.3, rng, residual=place)
    assert torch.equal(bits(place), bits(ln64.stream(x, r, 0.3, RNG)))
    if not x32:
        place = xd.clone()
        sq.dropout_add(place, place, 0.3, rng)
        assert torch.equal(bits(place), bits(ln64.stream(x, None, 0.3, RNG)))


def test_dropout_keeps_its_share():
    # 2^22 independent draws: five standard deviations
    n = 2**22
    x = torch.ones((1024, 4096), dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(x)
    seen = []
    for seed, p in ((1, 0.1), (1, 0.5), (2, 0.5), (2**63 - 1, 0.9)):
        sq.dropout_add(x, out, p, rng_tensor((seed, 0)))
        share = float((out == 0).double().mean())
        assert abs(share - p) <= 5 * (p * (1 - p) / n) ** 0.5
        seen.append(out == 0)
    # other seeds are independent: they agree where both drop or both keep
    both = float((seen[1] & seen[2]).double().mean())
    assert abs(both - 0.25) <= 5 * (0.25 * 0.75 / n) ** 0.5
    # rows and neighbouring columns too
    for a, b in ((seen[1][:-1], seen[1][1:]), (seen[1][:, :-1], seen[1][:, 1:]), (seen[1][:, :-4], seen[1][:, 4:])):
        assert abs(float((a & b).double().mean()) - 0.25) <= 6 * (0.25 * 0.75 / n) ** 0.5


def test_known_words():
    # the published test vectors of Philox4x32-10: of zeros, of ones, of pi's digits
    vectors = [((0, 0), (0, 0, 0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
               ((0xFFFFFFFF,) * 2, (0xFFFFFFFF,) * 4, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
               ((0xA4093822, 0x299F31D0), (0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344),
                (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))]
    signed = lambda v: v - 2**64 if v >= 2**63 else v
    # only the first has a place in a tensor that fits: word j is below p * 2^32 exactly where p says so
    key, counter, words = vectors[0]
    x = torch.ones((1, 4), device=DEV)
    for j, word in enumerate(words):
        for p in (np.nextafter(np.float32(word / 2**32), np.float32(0)), np.nextafter(np.float32(word / 2**32), np.float32(1))):
            out = torch.empty((1, 4), dtype=torch.bfloat16, device=DEV)
            sq.dropout_add(x, out, float(p), torch.tensor([signed(key[0] | key[1] << 32), 0], device=DEV))
            assert (float(out[0, j]) == 0) == (word < round(float(p) * 2**32))
    # the oracle's words against all of them
    for key, counter, words in vectors:
        c, k = list(counter), list(key)
        for _ in range(10):
            a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
            c = [(b >> 32) ^ c[1] ^ k[0], b % 2**32, (a >> 32) ^ c[3] ^ k[1], a % 2**32]
            k = [(k[0] + 0x9E3779B9) % 2**32, (k[1] + 0xBB67AE85) % 2**32]
        assert tuple(c) == words


def test_side_stream_and_graph():
    x, r, w, b = inputs(64, 1024, False, True, seed=8)
    dy, h, _, mean, rstd, d_h = bwd_inputs(64, 1024, False, True, seed=9)
    p = 0.2
    steps = [(7, 1), (7, 2), (-5, 2**62)]
    xd, rd, wd, bd = (t.to(DEV) for t in (x, r, w, b))
    back = [t.to(DEV) for t in (dy, h, w, mean, rstd)]
    new = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device=DEV)
    q, s = new(64, 1024, dtype=torch.int8), new(64, 8, dtype=torch.float32)
    hh, dx, drop, out = (new(64, 1024) for _ in range(4))
    dw, db = new(1024, dtype=torch.float32), new(1024, dtype=torch.float32)
    dhd, rng = d_h.to(DEV), rng_tensor(steps[0])
    ws = sq.layer_norm_bwd_workspace(64, 1024, DEV)
    outs = (q, s, hh, dx, drop, dw, db, out)

    def calls():
        sq.layer_norm_quant(xd, wd, bd, q, s, residual=rd, h=hh, p=p, rng=rng, offset=1)
        sq.layer_norm_bwd(*back, dx, dw=dw, db=db, d_h=dhd, dx_drop=drop, workspace=ws, p=p, rng=rng, offset=1)
        sq.dropout_add(xd, out, p, rng, residual=rd, offset=2)

    def taken():
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        return got

    want = []
    for st in steps:
        rng.copy_(torch.tensor(st))
        calls()
        want.append(taken())
        assert torch.equal(want[-1][2].cpu(), ln64.stream(x, r, p, st, 1))
        assert torch.equal(want[-1][7].cpu(), ln64.stream(x, r, p, st, 2))
    same = lambda a, b: all(torch.equal(u, v) for u, v in zip(a, b))
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        calls()
    assert same(taken(), want[-1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for i in (0, 1, 2, 0):  # the numbers are read when the graph runs
        rng.copy_(torch.tensor(steps[i]))
        graph.replay()
        assert same(taken(), want[i])
        calls()
        assert same(taken(), want[i])
