"""The layer norm, the dropout and the gated projection in 64 bits, on the CPU.
Shares no code with the library."""

import numpy as np
import torch


def kept(rng, T, D, p, offset=0):
    """Which elements of [T, D] a dropout keeps: Philox4x32-10 in Python's numpy, 64-bit words."""
    seed, step = (int(v) % 2**64 for v in rng)
    step = (step + offset) % 2**64
    mask = np.uint64(0xFFFFFFFF)
    blocks = -(-D // 4)
    c = [np.broadcast_to(np.arange(blocks, dtype=np.uint64), (T, blocks)),
         np.broadcast_to(np.arange(T, dtype=np.uint64)[:, None], (T, blocks)),
         np.full((T, blocks), step % 2**32, np.uint64), np.full((T, blocks), step >> 32, np.uint64)]
    k = [seed % 2**32, seed >> 32]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        s = np.uint64(32)
        c = [(b >> s) ^ c[1] ^ np.uint64(k[0]), b & mask, (a >> s) ^ c[3] ^ np.uint64(k[1]), a & mask]
        k = [(k[0] + 0x9E3779B9) % 2**32, (k[1] + 0xBB67AE85) % 2**32]
    words = np.stack(c, 2).reshape(T, -1)[:, :D]
    return torch.from_numpy(words >= np.uint64(round(float(np.float32(p)) * 2**32)))


def scale(p):
    """1 / (1 - p) of the fp32 p, rounded to fp32."""
    return float(np.float32(1.0 / (1.0 - float(np.float32(p)))))


def stream(x, residual=None, p=0.0, rng=None, offset=0):
    """bf16(residual + dropout(x)): one fp32 product, one fp32 sum."""
    v = x.float()
    if p > 0:
        v = torch.where(kept(rng, *x.shape, p, offset), v * scale(p), torch.zeros(()))
    if residual is not None:
        v = residual.float() + v
    return v.to(torch.bfloat16)


def norm(h, weight, bias, eps):
    """mean, rstd, y before rounding, and the magnitudes y is made of."""
    hd = h.double()
    mean = hd.mean(1)
    d = hd - mean[:, None]
    rstd = (d.square().mean(1) + eps) ** -0.5
    y = d * rstd[:, None] * weight.double()
    b = bias.double() if bias is not None else torch.zeros_like(y[0])
    return mean, rstd, y + b, y.abs() + b.abs()


def norm_bwd(dy, h, weight, mean, rstd, d_h=None):
    """dx, dw and db in 64 bits, each with the sum of the magnitudes it is made of."""
    r = rstd.double()[:, None]
    m = mean.double()[:, None]
    n = (h.double() - m) * r
    big_n = (h.double().abs() + m.abs()) * r  # n's own roundings are relative to these
    dy = dy.double()
    g = dy * weight.double()
    dx = r * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    size = r * (g.abs() + g.abs().mean(1, keepdim=True) + big_n * (g * big_n).abs().mean(1, keepdim=True))
    if d_h is not None:
        dx, size = dx + d_h.double(), size + d_h.double().abs()
    return dx, size, (dy * n).sum(0), (dy * big_n).abs().sum(0), dy.sum(0), dy.abs().sum(0)
