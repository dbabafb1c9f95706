"""Refusals of the norm and microscaled operators: bad arguments return their
code, or raise ValueError, before any device is touched (CPU only)."""

import pytest
import torch

import swiglu_backward_int8_amd as sq

BASE = 1 << 40  # fake addresses, never dereferenced: every call below is refused


@pytest.fixture(scope="module")
def lib():
    return sq.lib()


def caller(fn, names, ok):
    def call(**kw):
        args = list(ok)
        for k, v in kw.items():
            args[names.index(k)] = v
        return fn(*args)

    return call


def at(i):
    return BASE + (i << 30)


def test_rms_norm_quant_rejects_bad_arguments(lib):
    names = "x x_dtype residual weight y_q y_s y_bf16 h rstd T D group fmt eps stream".split()
    call = caller(lib.rms_norm_quant, names,
                  (at(0), 1, at(1), at(2), at(3), at(4), at(5), at(6), at(7), 8, 256, 128, 0, 1e-6, None))
    assert call(group=16) == 3 and call(group=256) == 3
    assert call(T=-1) == 2 and call(D=-1) == 2 and call(D=(1 << 22) + 1) == 2 and call(T=(1 << 31) + 1) == 2
    assert call(x_dtype=2) == 2 and call(fmt=2) == 2
    assert call(eps=-1.0) == 2 and call(eps=float("nan")) == 2 and call(eps=float("inf")) == 2
    assert call(x=None) == 1 and call(weight=None) == 1 and call(y_q=None) == 1 and call(y_s=None) == 1
    assert call(y_q=None, y_s=None, y_bf16=None) == 1
    for k in ("x", "residual", "weight", "y_q", "y_bf16", "h"):
        assert call(**{k: at(names.index(k)) + 8}) == 4, k
    assert call(y_s=at(4) + 2) == 4 and call(rstd=at(7) + 1) == 4
    assert call(y_q=at(0) + 64) == 5 and call(h=at(0)) == 5 and call(y_bf16=at(6)) == 5 and call(rstd=at(2)) == 5
    assert call(h=at(1) + 16) == 5  # the residual's place, but not the residual itself
    assert call(T=0, x=None, weight=None) == 0 and call(D=0, x=None) == 0


def test_rms_norm_bwd_rejects_bad_arguments(lib):
    names = "dy dy_dtype h weight rstd d_h dx dw ws ws_bytes T D stream".split()
    need = lib.rms_norm_bwd_workspace_bytes(8, 256)
    assert need >= 4 * 256 and lib.rms_norm_bwd_workspace_bytes(0, 256) == 0
    assert lib.rms_norm_bwd_workspace_bytes(-1, 256) == -1 and lib.rms_norm_bwd_workspace_bytes(8, (1 << 22) + 1) == -1
    call = caller(lib.rms_norm_bwd, names, (at(0), 1, at(1), at(2), at(3), at(4), at(5), at(6), at(7), need, 8, 256, None))
    assert call(T=-1) == 2 and call(D=(1 << 22) + 1) == 2 and call(dy_dtype=3) == 2
    assert call(ws_bytes=need - 1) == 2 and call(ws_bytes=-1) == 2
    for k in ("dy", "h", "weight", "rstd", "dx", "ws"):
        assert call(**{k: None}) == 1, k
    for k in ("dy", "h", "weight", "d_h", "dx", "ws"):
        assert call(**{k: at(("dy", "_", "h", "weight", "rstd", "d_h", "dx", "dw", "ws").index(k)) + 4}) == 4, k
    assert call(rstd=at(3) + 2) == 4 and call(dw=at(6) + 2) == 4
    assert call(dx=at(0) + 16) == 5 and call(dw=at(7)) == 5 and call(ws=at(1)) == 5 and call(dx=at(4) + 16) == 5
    assert call(T=0, D=0, dy=None) == 0 and call(T=0, dw=None, dy=None) == 0
    # a wide row needs the workspace even without dw
    wide = lib.rms_norm_bwd_workspace_bytes(8, 20000)
    assert call(D=20000, dw=None, ws=None, ws_bytes=wide) == 1 and call(D=20000, dw=None, ws_bytes=16) == 2


def test_mxfp4_quant_rejects_bad_arguments(lib):
    names = "x q s q_t s_t R K stream".split()
    call = caller(lib.mxfp4_quant, names, (at(0), at(1), at(2), at(3), at(4), 64, 96, None))
    assert call(R=-1) == 2 and call(K=-1) == 2 and call(K=(1 << 22) + 1) == 2 and call(R=(1 << 31) + 1) == 2
    assert call(x=None) == 1 and call(q=None) == 1 and call(s=None) == 1 and call(q_t=None) == 1 and call(s_t=None) == 1
    assert call(q=None, s=None, q_t=None, s_t=None) == 1
    assert call(x=at(0) + 2) == 4 and call(q=at(1) + 8) == 4 and call(q_t=at(3) + 8) == 4
    assert call(q=at(0) + 128) == 5 and call(s=at(1)) == 5 and call(s_t=at(2)) == 5 and call(q_t=at(1) + 16) == 5
    assert call(R=0, x=None) == 0 and call(K=0, x=None) == 0


def test_mxfp4_gemm_rejects_bad_arguments(lib):
    names = "A sA B sB C M N K out stream".split()
    call = caller(lib.mxfp4_gemm, names, (at(0), at(1), at(2), at(3), at(4), 64, 96, 128, 0, None))
    assert call(M=-1) == 2 and call(N=-1) == 2 and call(K=-32) == 2 and call(K=48) == 2 and call(K=(1 << 22) + 32) == 2
    assert call(out=2) == 2 and call(M=1 << 31, N=1 << 31) == 2 and call(M=(1 << 31) + 1) == 2
    for k in ("A", "sA", "B", "sB", "C"):
        assert call(**{k: None}) == 1, k
    assert call(A=at(0) + 8) == 4 and call(B=at(2) + 4) == 4 and call(C=at(4) + 2) == 4 and call(C=at(4) + 1, out=1) == 4
    assert call(C=at(0) + 16) == 5 and call(C=at(1)) == 5 and call(C=at(2)) == 5 and call(C=at(3)) == 5
    assert call(M=0, A=None, C=None) == 0 and call(N=0, B=None, C=None) == 0


def test_dequant_rejects_bad_arguments(lib):
    f = lib.mxfp4_dequant
    assert f(at(0), at(1), at(2), -1, 64, None) == 2 and f(at(0), at(1), at(2), 4, (1 << 22) + 1, None) == 2
    assert f(None, at(1), at(2), 4, 64, None) == 1 and f(at(0), None, at(2), 4, 64, None) == 1
    assert f(at(0), at(1), None, 4, 64, None) == 1
    assert f(at(0) + 8, at(1), at(2), 4, 64, None) == 4 and f(at(0), at(1), at(2) + 2, 4, 64, None) == 4
    assert f(at(0), at(1), at(0) + 16, 4, 64, None) == 5 and f(at(0), at(2) + 7, at(2), 4, 64, None) == 5
    assert f(None, None, None, 0, 64, None) == 0
    f = lib.group_dequant
    assert f(at(0), at(1), at(2), 4, 64, 48, 0, None) == 3
    assert f(at(0), at(1), at(2), 4, -64, 32, 0, None) == 2 and f(at(0), at(1), at(2), 4, 64, 32, 2, None) == 2
    assert f(at(0), at(1), at(2), 4, (1 << 23) + 1, 32, 0, None) == 2
    assert f(None, at(1), at(2), 4, 64, 32, 0, None) == 1 and f(at(0), at(1) + 2, at(2), 4, 64, 32, 0, None) == 4
    assert f(at(0), at(1), at(1), 4, 64, 32, 0, None) == 5
    assert f(None, None, None, 4, 0, 32, 0, None) == 0


def test_binding_rejects_tensors_on_the_host():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w, q, s = x[0].clone(), torch.zeros((4, 64), dtype=torch.int8), torch.zeros((4, 1))
    u = torch.zeros((4, 32), dtype=torch.uint8)
    e = torch.zeros((4, 2), dtype=torch.uint8)
    for call in (lambda: sq.rms_norm_quant(x, w, q, s), lambda: sq.rms_norm_bwd(x, x, w, s[:, 0], x),
                 lambda: sq.mxfp4_quant(x, u, e), lambda: sq.mxfp4_gemm(u, e, u, e, s),
                 lambda: sq.mxfp4_dequant(u, e, x), lambda: sq.group_dequant(q, s, x)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_binding_rejects_bad_tensors():
    d = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype, device="cuda:0")
    f32, i8, u8 = torch.float32, torch.int8, torch.uint8
    x, w, q, s = d(4, 64), d(64), d(4, 64, dtype=i8), d(4, 1, dtype=f32)
    u, e = d(4, 32, dtype=u8), d(4, 2, dtype=u8)
    sq.rms_norm_quant(x, w, q, s)  # what the refused calls below vary
    sq.mxfp4_gemm(u, e, u, e, d(4, 4))
    bad = [
        lambda: sq.rms_norm_quant(x[0], w, q, s),                      # rank
        lambda: sq.rms_norm_quant(x.half(), w, q, s),                  # type
        lambda: sq.rms_norm_quant(x, d(32), q, s),                     # shape
        lambda: sq.rms_norm_quant(x, w, d(4, 64, dtype=torch.int16), s),
        lambda: sq.rms_norm_quant(x, w, q, s, group_size=48),
        lambda: sq.rms_norm_quant(x, w, q),                            # codes without scales
        lambda: sq.rms_norm_quant(x, w),                               # no output
        lambda: sq.rms_norm_quant(x, w, q, s, residual=d(64, 4).t()),  # not contiguous
        lambda: sq.rms_norm_quant(x, w, q, s, h=x),                    # over an input
        lambda: sq.rms_norm_quant(x, w, q, s, rstd=d(4, 1, dtype=f32)),
        lambda: sq.rms_norm_bwd(x, d(4, 64), w, d(4, dtype=f32), d(4, 64), dw=d(64, dtype=f32)),  # no workspace
        lambda: sq.rms_norm_bwd(x, d(4, 64), w, d(4, dtype=f32), d(4, 64), dw=d(64, dtype=f32),
                                workspace=d(8, dtype=u8)),             # too small
        lambda: sq.rms_norm_bwd(x, d(4, 64), w, d(4, dtype=f32), x),
        lambda: sq.mxfp4_quant(x, u),
        lambda: sq.mxfp4_quant(x, u, e, q_t=d(64, 16, dtype=u8)),
        lambda: sq.mxfp4_quant(x, d(4, 16, dtype=u8), e),
        lambda: sq.mxfp4_quant(x),
        lambda: sq.mxfp4_gemm(u, e, d(4, 16, dtype=u8), e, d(4, 4)),   # another K
        lambda: sq.mxfp4_gemm(d(4, 24, dtype=u8), e, u, e, d(4, 4)),
        lambda: sq.mxfp4_gemm(u, e, u, e, d(4, 5)),
        lambda: sq.mxfp4_gemm(u, e, u, e, d(4, 4, dtype=i8)),
        lambda: sq.mxfp4_dequant(u, e, d(4, 96)),
        lambda: sq.mxfp4_dequant(u, e.cpu(), d(4, 64)),
        lambda: sq.group_dequant(q, s, d(4, 64, dtype=f32)),
        lambda: sq.group_dequant(q, s, d(4, 64), group_size=32),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("case %d was taken" % i, flush=True)
