"""The row operators in 64 bits, on the CPU: the RMS norm and its gradients, the
group quantiser in its own fp32 steps (numpy), and the microscaled 4-bit format
from its definition.  Shares no code with the library."""

import numpy as np
import torch

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def norm(x, residual, weight, eps):
    """h (bf16), and rstd and y before rounding in 64 bits."""
    h = x.float() if residual is None else x.float() + residual.float()
    h = h.to(torch.bfloat16)
    hd = h.double()
    rstd = (hd.square().mean(1) + eps) ** -0.5
    return h, rstd, hd * rstd[:, None] * weight.double()


def norm_bwd(dy, h, weight, rstd, d_h=None):
    """dx and dw in 64 bits, and the sums of the magnitudes they are made of."""
    n = h.double() * rstd.double()[:, None]
    dy = dy.double()
    g = dy * weight.double()
    r = rstd.double()[:, None]
    dx = r * (g - n * (g * n).mean(1, keepdim=True))
    size = r * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if d_h is not None:
        dx, size = dx + d_h.double(), size + d_h.double().abs()
    return dx, size, (dy * n).sum(0), (dy * n).abs().sum(0)


def group_quant(y, group, e4m3):
    """Codes (bytes) and scales of bf16 rows y, every step one fp32 operation."""
    R, K = y.shape
    v = np.zeros((R, -(-K // group) * group), np.float32)
    v[:, :K] = y.float().numpy()
    g = v.reshape(R, -1, group)
    amax = np.abs(g).max(2, keepdims=True)
    top = np.float32(448.0 if e4m3 else 127.0)
    scale = np.where(amax == 0, np.float32(1), amax / top).astype(np.float32)
    with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
        p = g * (np.float32(1) / scale)
    p = np.where(g == 0, g, np.clip(p, -top, top)).astype(np.float32)
    if e4m3:
        codes = torch.from_numpy(p).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    else:
        codes = np.rint(p).astype(np.int8).view(np.uint8)
    return codes.reshape(R, -1)[:, :K], scale[..., 0]


def mx_quant(x):
    """Packed E2M1 codes and E8M0 bytes of bf16 rows x."""
    R, K = x.shape
    blocks = -(-K // 32)
    v = np.zeros((R, blocks * 32))
    v[:, :K] = x.double().numpy()
    v = v.reshape(R, blocks, 32)
    amax = np.abs(v).max(2)
    finite = np.isfinite(v).all(2)
    e = np.where((amax > 0) & finite, np.frexp(np.where(finite, amax, 1.0))[1] - 1 - 2, 0)
    e = np.maximum(e, -127)
    a = np.abs(np.where(finite[..., None], v, 0.0)) * 2.0 ** -e[..., None].astype(np.float64)
    d = np.abs(a[..., None] - LEVELS)                       # distance to every level
    near = d == d.min(-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))  # a tie goes to the even code
    code = (code | (np.signbit(v) << 3)).astype(np.uint8).reshape(R, -1)
    return code[:, 0::2] | code[:, 1::2] << 4, np.where(finite, e + 127, 255).astype(np.uint8)


def mx_values(q, s):
    """The values of packed codes, in 64 bits (NaN where the exponent is 255)."""
    code = np.stack([q & 15, q >> 4], 2).reshape(q.shape[0], -1)
    v = np.where(code >= 8, -1.0, 1.0) * LEVELS[code & 7]
    e = np.repeat(s.astype(np.float64) - 127, 32, 1)
    return np.where(np.repeat(s, 32, 1) == 255, np.nan, v * 2.0**e)
