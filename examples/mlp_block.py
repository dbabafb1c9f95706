"""One pre-norm SwiGLU block through the library, in 8, 4 and 16 bits.

    h   = x + residual;  y = h / rms(h) * w          rms_norm_quant
    [gate | up] = y . Wgu^T                          i8_gemm_group_scaled, or mxfp4_gemm
    a   = silu(gate) * up                            silu_fwd_quant
    out = a . Wd^T                                   i8_gemm_group_scaled, or mxfp4_gemm

``forward_int8`` is the serving path: the norm and SwiGLU write the int8 codes
that the next product reads.  ``train_mxfp4`` is a training step: mxfp4_quant
codes every operand along both axes in one read, so that each of the three
products of a linear layer contracts over blocks of its own axis; the SwiGLU
backward pass's int8 codes come back through group_dequant; rms_norm_bwd takes
the dgrad product's output and joins the residual's gradient.

``train_bf16`` is a training step in bf16, with a layer norm and two dropouts:

    h   = residual + dropout(x);  y = (h - mean) / std(h) * w + b    layer_norm_quant
    a   = silu(y . Wg^T) * (y . Wu^T)                                swiglu_gemm
    out = dropout(a) . Wd^T                                          dropout_add, torch's product

Its masks are never stored: the backward pass makes them again from the same
numbers (rng), which lie on the device, so a captured step can change them.  A mask
is told by the sum of the step's number and the call's offset, so the dropouts of a
step lie 2^32 apart: a step's second mask is none that a later step draws.

    python examples/mlp_block.py [T D H]

prints how far each result is from the same block in fp32 (an MXFP4 code is
within about an eighth of its value, so the 4-bit results are that coarse).
"""

import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import swiglu_backward_int8_amd as sq  # noqa: E402

EPS = 1e-6
NORM, ACTIVATION = 0 << 32, 1 << 32  # offsets of a step's dropouts (layer l of a model: 2 * l << 32 and 2 * l + 1 << 32)


class Mx:
    """A bf16 matrix as microscaled 4-bit codes: by rows, and by columns where asked."""

    def __init__(self, x, columns=False):
        new = lambda shape: torch.empty(shape, dtype=torch.uint8, device=x.device)
        R, K = x.shape
        self.q, self.s = map(new, sq.mxfp4_shapes(R, K))
        self.q_t, self.s_t = map(new, sq.mxfp4_shapes(K, R)) if columns else (None, None)
        sq.mxfp4_quant(x, self.q, self.s, q_t=self.q_t, s_t=self.s_t)

    @property
    def rows(self):
        return self.q, self.s

    @property
    def cols(self):
        return self.q_t, self.s_t


def product(a, b, dtype=torch.bfloat16):
    C = torch.empty((a[0].shape[0], b[0].shape[0]), dtype=dtype, device=a[0].device)
    sq.mxfp4_gemm(*a, *b, C)
    return C


def int8_blocks(W):
    """A weight [N, K] in int8 with a scale per 128 x 128 block (N and K multiples of 128)."""
    N, K = W.shape
    b = W.float().view(N // 128, 128, K // 128, 128)
    s = b.abs().amax((1, 3)) / 127.0
    q = torch.round(b / s[:, None, :, None]).clamp(-127, 127).view(N, K).to(torch.int8)
    return q, s.contiguous()


def norm(x, residual, w, codes=False):
    T, D = x.shape
    new = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device=x.device)
    h, rstd = new(T, D, dtype=torch.bfloat16), new(T, dtype=torch.float32)
    if codes:
        q, s = new(T, D, dtype=torch.int8), new(T, -(-D // 128), dtype=torch.float32)
        sq.rms_norm_quant(x, w, q, s, residual=residual, h=h, rstd=rstd, eps=EPS)
        return h, rstd, (q, s)
    y = new(T, D, dtype=torch.bfloat16)
    sq.rms_norm_quant(x, w, residual=residual, h=h, rstd=rstd, y_bf16=y, eps=EPS)
    return h, rstd, y


def forward_int8(x, residual, w, Wgu, Wd):
    """Wgu, Wd: (codes, scales) of int8_blocks.  Returns out and the new residual stream."""
    T, H = x.shape[0], Wd[0].shape[1]
    new = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device=x.device)
    h, _, y = norm(x, residual, w, codes=True)
    gu = new(T, 2 * H, dtype=torch.bfloat16)
    sq.i8_gemm_group_scaled(*y, *Wgu, gu, b_rows_per_scale=128)
    a, s = new(T, H, dtype=torch.int8), new(T, H // 128, dtype=torch.float32)
    sq.silu_fwd_quant(gu, a, s)
    out = new(T, Wd[0].shape[0], dtype=torch.bfloat16)
    sq.i8_gemm_group_scaled(a, s, *Wd, out, b_rows_per_scale=128)
    return out, h


def train_mxfp4(x, residual, w, Wgu, Wd, d_out, d_h):
    """Forward and backward in 4 bits.  Wgu [2H, D], Wd [D, H] bf16; d_out, d_h the
    gradients of out and of the residual stream.  Returns out and the gradients
    of x (and residual), w, Wgu and Wd."""
    T, D = x.shape
    H = Wd.shape[1]
    new = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device=x.device)
    wgu, wd = Mx(Wgu, columns=True), Mx(Wd, columns=True)

    h, rstd, y = norm(x, residual, w)
    my = Mx(y, columns=True)
    gu = product(my.rows, wgu.rows)
    a = new(T, H, dtype=torch.bfloat16)
    sq.silu_fwd_quant(gu, new(T, H, dtype=torch.int8), new(T, -(-H // 128), dtype=torch.float32), y_bf16=a)
    ma = Mx(a, columns=True)
    out = product(ma.rows, wd.rows)

    mo = Mx(d_out, columns=True)
    d_a = product(mo.rows, wd.cols)                        # over D
    d_Wd = product(mo.cols, ma.cols, torch.float32)        # over tokens
    dgu_q, dgu_s, a_q, a_s = sq.empty_outputs(T, H, x.device)
    sq.silu_dot_fwd_bwd_quant_fuse(gu, d_a, dgu_q, dgu_s, a_q, a_s)
    d_gu = new(T, 2 * H, dtype=torch.bfloat16)
    sq.group_dequant(dgu_q, dgu_s, d_gu)
    mg = Mx(d_gu, columns=True)
    d_y = product(mg.rows, wgu.cols, torch.float32)        # over 2H
    d_Wgu = product(mg.cols, my.cols, torch.float32)       # over tokens
    d_x, d_w = new(T, D, dtype=torch.bfloat16), new(D, dtype=torch.float32)
    sq.rms_norm_bwd(d_y, h, w, rstd, d_x, dw=d_w, d_h=d_h, workspace=sq.rms_norm_bwd_workspace(T, D, x.device))
    return out, d_x, d_w, d_Wgu, d_Wd


def train_bf16(x, residual, w, b, Wgu, Wd, d_out, d_h, p, rng):
    """Forward and backward in bf16.  rng: int64 [2], a seed and the step's number
    (below 2^32).  Returns out and the gradients of x, residual, w, b, Wgu and Wd."""
    T, D = x.shape
    H = Wd.shape[1]
    new = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device=x.device)
    h, y, mean, rstd = new(T, D), new(T, D), new(T, dtype=torch.float32), new(T, dtype=torch.float32)
    sq.layer_norm_quant(x, w, b, residual=residual, h=h, mean=mean, rstd=rstd, y_bf16=y, eps=EPS, p=p, rng=rng,
                        offset=NORM)
    a, gu, ad = new(T, H), new(T, 2 * H), new(T, H)
    sq.swiglu_gemm(y, Wgu, a, gu=gu)
    sq.dropout_add(a, ad, p, rng, offset=ACTIVATION)
    out = ad @ Wd.t()

    d_Wd = d_out.t() @ ad
    d_a = d_out @ Wd
    sq.dropout_add(d_a, d_a, p, rng, offset=ACTIVATION)
    d_y, d_Wgu = new(T, D), new(2 * H, D)
    sq.swiglu_gemm_bwd(d_a, gu, y, Wgu, gu, dx=d_y, dw=d_Wgu, workspace=sq.swiglu_gemm_bwd_workspace(T, H, D, x.device))
    d_residual, d_x = new(T, D), new(T, D) if p > 0 else None
    d_w, d_b = new(D, dtype=torch.float32), new(D, dtype=torch.float32)
    sq.layer_norm_bwd(d_y, h, w, mean, rstd, d_residual, dw=d_w, db=d_b, d_h=d_h, dx_drop=d_x,
                      workspace=sq.layer_norm_bwd_workspace(T, D, x.device), p=p, rng=rng, offset=NORM)
    return out, d_residual if d_x is None else d_x, d_residual, d_w, d_b, d_Wgu, d_Wd


def reference_bf16(x, residual, w, b, Wgu, Wd, d_out, d_h, p, rng):
    """The same in fp32 through autograd, with the library's masks."""
    def mask(rows, cols, offset):
        m = torch.empty((rows, cols), dtype=torch.bfloat16, device=x.device)
        sq.dropout_add(torch.ones_like(m), m, p, rng, offset=offset)
        return (m > 0).float() / (1 - p)

    T, D = x.shape
    H = Wd.shape[1]
    x, residual, w, b, Wgu, Wd = leaves = [t.float().requires_grad_() for t in (x, residual, w, b, Wgu, Wd)]
    h = residual + x * mask(T, D, NORM)
    c = h - h.mean(1, keepdim=True)
    y = c * torch.rsqrt(c.square().mean(1, keepdim=True) + EPS) * w + b
    gate, up = (y @ Wgu.t()).chunk(2, 1)
    out = (torch.nn.functional.silu(gate) * up * mask(T, H, ACTIVATION)) @ Wd.t()
    torch.autograd.backward([out, h], [d_out.float(), d_h.float()])
    return [out.detach()] + [t.grad for t in leaves]


def reference(x, residual, w, Wgu, Wd, d_out, d_h):
    x, w, Wgu, Wd = (t.float().requires_grad_() for t in (x, w, Wgu, Wd))
    h = x + residual.float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * w
    gate, up = (y @ Wgu.t()).chunk(2, 1)
    out = (torch.nn.functional.silu(gate) * up) @ Wd.t()
    torch.autograd.backward([out, h], [d_out.float(), d_h.float()])
    return out.detach(), h.detach(), x.grad, w.grad, Wgu.grad, Wd.grad


def main(T=512, D=1024, H=1408, device="cuda:0"):
    """Runs both and returns {name: relative error}."""
    g = torch.Generator(device=device).manual_seed(0)
    rand = lambda *shape, std=1.0: (torch.randn(shape, generator=g, device=device) * std).bfloat16()
    x, residual, w = rand(T, D), rand(T, D), (1 + rand(D, std=0.1).float()).bfloat16()
    Wgu, Wd = rand(2 * H, D, std=D**-0.5), rand(D, H, std=H**-0.5)
    d_out, d_h = rand(T, D, std=0.01), rand(T, D, std=0.01)
    want = reference(x, residual, w, Wgu, Wd, d_out, d_h)
    far = lambda a, b: float((a.float() - b).norm() / b.norm())
    out8, h8 = forward_int8(x, residual, w, int8_blocks(Wgu), int8_blocks(Wd))
    got = train_mxfp4(x, residual, w, Wgu, Wd, d_out, d_h)
    errors = {"int8 out": far(out8, want[0]), "int8 h": far(h8, want[1])}
    errors.update(zip(("mxfp4 out", "mxfp4 d_x", "mxfp4 d_w", "mxfp4 d_Wgu", "mxfp4 d_Wd"),
                      (far(a, b) for a, b in zip(got, (want[0],) + want[2:]))))
    rng = torch.tensor([2024, 7], device=device)
    args = x, residual, w, rand(D, std=0.1), Wgu, Wd, d_out, d_h, 0.1, rng
    names = "out d_x d_residual d_w d_b d_Wgu d_Wd".split()
    errors.update(("bf16 " + n, far(a, b)) for n, a, b in zip(names, train_bf16(*args), reference_bf16(*args)))
    return errors


if __name__ == "__main__":
    for name, err in main(*map(int, sys.argv[1:4])).items():
        print("%-12s %.4f" % (name, err))
