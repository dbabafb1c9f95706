"""Refusals of the layer norm, the dropout and the gated projection: bad arguments
return their code, or raise ValueError, before any device is touched (CPU only)."""

import pytest
import torch

import swiglu_backward_int8_amd as sq
from test_operators_abi import at, caller

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    return sq.lib()


def test_layer_norm_quant_rejects_bad_arguments(lib):
    names = "x x_dtype residual weight bias y_q y_s y_bf16 h mean rstd T D group fmt eps p rng offset stream".split()
    call = caller(lib.layer_norm_quant, names,
                  (at(0), 1, at(1), at(2), at(3), at(4), at(5), at(6), at(7), at(8), at(9), 8, 256, 128, 0, 1e-5, 0.1, at(10), 0, None))
    assert call(group=16) == 3 and call(group=256) == 3
    assert call(T=-1) == 2 and call(D=-1) == 2 and call(D=(1 << 22) + 1) == 2 and call(T=(1 << 31) + 1) == 2
    assert call(x_dtype=2) == 2 and call(fmt=2) == 2
    assert call(eps=-1.0) == 2 and call(eps=NAN) == 2 and call(eps=INF) == 2
    assert call(p=-0.1) == 2 and call(p=1.0) == 2 and call(p=NAN) == 2 and call(p=1 - 2.0**-26) == 2  # fp32's 1
    for k in ("x", "weight", "y_q", "y_s", "rng"):
        assert call(**{k: None}) == 1, k
    assert call(y_q=None, y_s=None, y_bf16=None) == 1
    pointers = [n for n in names if n in "x residual weight bias y_q y_s y_bf16 h mean rstd rng".split()]
    place = {n: at(i) for i, n in enumerate(pointers)}
    for k in ("x", "residual", "weight", "bias", "y_q", "y_bf16", "h"):
        assert call(**{k: place[k] + 8}) == 4, k
    for k in ("y_s", "mean", "rstd"):
        assert call(**{k: place[k] + 2}) == 4, k
    assert call(rng=place["rng"] + 4) == 4
    for out in ("y_q", "y_s", "y_bf16", "h", "mean", "rstd"):
        for other in pointers:
            if other != out and (out, other) != ("h", "residual"):
                assert call(**{out: place[other]}) == 5, (out, other)
    assert call(h=at(1) + 16) == 5  # the residual's place, but not the residual itself
    assert call(T=0, x=None, weight=None, rng=None) == 0 and call(D=0, x=None) == 0


def test_layer_norm_bwd_rejects_bad_arguments(lib):
    names = "dy dy_dtype h weight mean rstd d_h dx dx_drop dw db ws ws_bytes T D p rng offset stream".split()
    need = lib.layer_norm_bwd_workspace_bytes(8, 256)
    assert need >= 8 * 256 and lib.layer_norm_bwd_workspace_bytes(0, 256) == 0
    assert lib.layer_norm_bwd_workspace_bytes(-1, 256) == -1 and lib.layer_norm_bwd_workspace_bytes(8, (1 << 22) + 1) == -1
    call = caller(lib.layer_norm_bwd, names, (at(0), 1, at(1), at(2), at(3), at(4), at(5), at(6), at(7), at(8), at(9), at(10), need, 8, 256,
                                              0.1, at(11), 0, None))
    pointers = "dy h weight mean rstd d_h dx dx_drop dw db ws rng".split()
    place = {n: at(i) for i, n in enumerate(pointers)}
    assert call(T=-1) == 2 and call(D=(1 << 22) + 1) == 2 and call(dy_dtype=3) == 2
    assert call(p=1.0) == 2 and call(p=NAN) == 2 and call(p=0.0) == 2  # dx_drop of no dropout
    assert call(ws_bytes=need - 1) == 2 and call(ws_bytes=-1) == 2
    for k in ("dy", "h", "weight", "mean", "rstd", "dx", "ws", "rng"):
        assert call(**{k: None}) == 1, k
    for k in ("dy", "h", "weight", "d_h", "dx", "dx_drop", "ws"):
        assert call(**{k: place[k] + 4}) == 4, k
    for k in ("mean", "rstd", "dw", "db"):
        assert call(**{k: place[k] + 2}) == 4, k
    assert call(rng=place["rng"] + 4) == 4
    for out in ("dx", "dx_drop", "dw", "db", "ws"):
        for other in pointers:
            if other != out and (out, other) != ("dx", "d_h"):
                assert call(**{out: place[other]}) == 5, (out, other)
    assert call(dx=at(5) + 16) == 5
    assert call(T=0, D=0, dy=None) == 0 and call(T=0, dw=None, db=None, dy=None) == 0
    assert call(T=0, dw=at(8) + 2) == 4 and call(T=0, db=at(8)) == 5
    # a wide row needs the workspace even without sums
    wide = lib.layer_norm_bwd_workspace_bytes(8, 20000)
    assert call(D=20000, dw=None, db=None, ws=None, ws_bytes=wide) == 1 and call(D=20000, dw=None, db=None, ws_bytes=16) == 2


def test_dropout_add_rejects_bad_arguments(lib):
    names = "x x_dtype residual out T D p rng offset stream".split()
    call = caller(lib.dropout_add, names, (at(0), 1, at(1), at(2), 8, 256, 0.1, at(3), 0, None))
    assert call(T=-1) == 2 and call(D=-1) == 2 and call(D=(1 << 22) + 1) == 2 and call(T=(1 << 31) + 1) == 2 and call(x_dtype=2) == 2
    assert call(T=1 << 31, D=1 << 22) == 2
    assert call(p=-0.1) == 2 and call(p=1.0) == 2 and call(p=NAN) == 2
    assert call(x=None) == 1 and call(out=None) == 1 and call(rng=None) == 1
    assert call(x=at(0) + 8) == 4 and call(residual=at(1) + 8) == 4 and call(out=at(2) + 8) == 4 and call(rng=at(3) + 4) == 4
    assert call(out=at(0) + 16) == 5 and call(out=at(1) + 16) == 5 and call(out=at(3)) == 5
    assert call(out=at(0), x_dtype=0) == 5  # fp32 x cannot be its own bf16 output
    assert call(T=0, x=None, out=None) == 0 and call(D=0, x=None) == 0


def test_swiglu_gemm_rejects_bad_arguments(lib):
    names = "x w y gu T H D stream".split()
    call = caller(lib.swiglu_gemm, names, (at(0), at(1), at(2), at(3), 8, 64, 256, None))
    for k in ("T", "H", "D"):
        assert call(**{k: -8}) == 2
    assert call(H=60) == 2 and call(D=252) == 2 and call(H=(1 << 20) + 8) == 2 and call(D=(1 << 20) + 8) == 2 and call(T=(1 << 31) + 1) == 2
    assert call(T=1 << 31, H=1 << 12) == 2  # more tiles than are counted
    for k in ("x", "w", "y"):
        assert call(**{k: None}) == 1, k
    for i, k in enumerate(("x", "w", "y", "gu")):
        assert call(**{k: at(i) + 8}) == 4, k
    for out in (2, 3):
        for i in range(4):
            if i != out:
                assert call(**{names[out]: at(i)}) == 5, (names[out], names[i])
    assert call(T=0, x=None, w=None, y=None) == 0 and call(H=0, y=None) == 0


def test_swiglu_gemm_bwd_rejects_bad_arguments(lib):
    names = "dy gu x w d_gu dx dx_dtype dw dw_dtype ws ws_bytes T H D stream".split()
    T, H, D = 64, 5504, 256  # few tiles over a long sum: slices
    need = lib.swiglu_gemm_bwd_workspace_bytes(T, H, D)
    assert need > 0 and need % 16 == 0
    assert lib.swiglu_gemm_bwd_workspace_bytes(0, H, D) == 0 and lib.swiglu_gemm_bwd_workspace_bytes(T, 60, D) == -1
    assert lib.swiglu_gemm_bwd_workspace_bytes(-1, H, D) == -1
    call = caller(lib.swiglu_gemm_bwd, names, (at(0), at(1), at(2), at(3), at(4), at(5), 1, at(6), 1, at(7), need, T, H, D, None))
    pointers = "dy gu x w d_gu dx dw ws".split()
    assert call(T=-1) == 2 and call(H=5500) == 2 and call(D=260) == 2 and call(dx_dtype=2) == 2 and call(dw_dtype=-1) == 2
    assert call(ws_bytes=need - 1) == 2 and call(ws_bytes=-1) == 2 and call(T=1 << 31, D=1 << 20) == 2
    for k in ("dy", "gu", "x", "w", "d_gu", "ws"):
        assert call(**{k: None}) == 1, k
    for i, k in enumerate(pointers):
        assert call(**{k: at(i) + 8}) == 4, k
    for out in ("d_gu", "dx", "dw", "ws"):
        for i, other in enumerate(pointers):
            if other != out and (out, other) != ("d_gu", "gu"):
                assert call(**{out: at(i)}) == 5, (out, other)
    assert call(d_gu=at(1) + 16) == 5  # gu's place, but not gu itself
    assert call(T=0, H=0, dy=None) == 0 and call(T=0, dw=None, dy=None) == 0


def test_binding_rejects_tensors_on_the_host():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w, q, s = x[0].clone(), torch.zeros((4, 64), dtype=torch.int8), torch.zeros((4, 1))
    rng = torch.zeros(2, dtype=torch.int64)
    W, gu = torch.zeros((128, 64), dtype=torch.bfloat16), torch.zeros((4, 128), dtype=torch.bfloat16)
    for call in (lambda: sq.layer_norm_quant(x, w, y_q=q, y_s=s), lambda: sq.layer_norm_bwd(x, x, w, s[:, 0], s[:, 0], x),
                 lambda: sq.dropout_add(x, x, 0.1, rng), lambda: sq.swiglu_gemm(x, W, x),
                 lambda: sq.swiglu_gemm_bwd(x, gu, x, W, gu)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_binding_rejects_bad_tensors():
    d = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype, device="cuda:0")
    f32, i8, i64 = torch.float32, torch.int8, torch.int64
    x, w, y, m = d(4, 64), d(64), d(4, 64), d(4, dtype=f32)
    rng, W, gu = d(2, dtype=i64), d(128, 64), d(4, 128)
    sq.layer_norm_quant(x, w, y_bf16=y, p=0.5, rng=rng)  # what the refused calls below vary
    sq.layer_norm_bwd(x, d(4, 64), w, m, d(4, dtype=f32), y, dx_drop=d(4, 64), p=0.5, rng=rng)
    sq.dropout_add(x, y, 0.5, rng)
    sq.swiglu_gemm(x, W, y, gu=gu)
    sq.swiglu_gemm_bwd(x, gu, d(4, 64), W, d(4, 128), dx=y)
    bad = [
        lambda: sq.layer_norm_quant(x[0], w, y_bf16=y),
        lambda: sq.layer_norm_quant(x.half(), w, y_bf16=y),
        lambda: sq.layer_norm_quant(x, d(32), y_bf16=y),
        lambda: sq.layer_norm_quant(x, w, bias=w.float(), y_bf16=y),
        lambda: sq.layer_norm_quant(x, w),
        lambda: sq.layer_norm_quant(x, w, y_q=d(4, 64, dtype=i8)),
        lambda: sq.layer_norm_quant(x, w, y_bf16=x),
        lambda: sq.layer_norm_quant(x, w, y_bf16=y, mean=d(4, 1, dtype=f32)),
        lambda: sq.layer_norm_quant(x, w, y_bf16=y, p=0.5),
        lambda: sq.layer_norm_quant(x, w, y_bf16=y, p=1.0, rng=rng),
        lambda: sq.layer_norm_quant(x, w, y_bf16=y, p=NAN, rng=rng),
        lambda: sq.layer_norm_quant(x, w, y_bf16=y, p=0.5, rng=rng.int()),
        lambda: sq.layer_norm_quant(x, w, y_bf16=y, p=0.5, rng=rng.cpu()),
        lambda: sq.layer_norm_quant(x, w, y_bf16=y, p=0.5, rng=rng, offset=2**63),
        lambda: sq.layer_norm_bwd(x, d(4, 64), w, m, m, y, dw=d(64, dtype=f32)),           # no workspace
        lambda: sq.layer_norm_bwd(x, d(4, 64), w, m, m, y, db=d(64, dtype=f32), workspace=d(8, dtype=i8)),
        lambda: sq.layer_norm_bwd(x, d(4, 64), w, m, m, x),
        lambda: sq.layer_norm_bwd(x, d(4, 64), w, m, m, y, dx_drop=d(4, 64)),             # of no dropout
        lambda: sq.layer_norm_bwd(x, d(4, 64), w, m, m, y, dx_drop=d(4, 64), p=0.5),
        lambda: sq.layer_norm_bwd(x, d(4, 64), w, m, m, y, p=2.0),
        lambda: sq.dropout_add(x, y, 0.5, None),
        lambda: sq.dropout_add(x, y, -0.5, rng),
        lambda: sq.dropout_add(x, d(4, 64, dtype=f32), 0.5, rng),
        lambda: sq.dropout_add(x, d(64, 4).t(), 0.5, rng),
        lambda: sq.dropout_add(x, y, 0.5, rng, residual=d(4, 32)),
        lambda: sq.swiglu_gemm(x, d(127, 64), y),
        lambda: sq.swiglu_gemm(x, d(120, 64), y),                                           # H = 60
        lambda: sq.swiglu_gemm(x, d(128, 32), y),
        lambda: sq.swiglu_gemm(x.float(), W, y),
        lambda: sq.swiglu_gemm(x, W, y, gu=y),
        lambda: sq.swiglu_gemm(x, W, x),
        lambda: sq.swiglu_gemm_bwd(x, gu, d(4, 64), W, d(4, 128), dx=d(4, 64, dtype=torch.float16)),
        lambda: sq.swiglu_gemm_bwd(x, gu, d(4, 64), W, d(4, 128), dw=d(64, 128)),
        lambda: sq.swiglu_gemm_bwd(x, gu, d(4, 64), W, d(4, 64)),
        lambda: sq.swiglu_gemm_bwd(x, gu, d(3, 64), W, d(4, 128)),
        lambda: sq.swiglu_gemm_bwd(d(64, 5504), d(64, 11008), d(64, 256), d(11008, 256), d(64, 11008), dx=d(64, 256)),  # no workspace
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("case %d was taken" % i, flush=True)
