"""The RMS norm and MXFP4 operators as they are measured: cases, inputs, the
plain form of each operator in elementary torch operations, the library's
calls, and the operators' definitions in 64 bits.

  rms_norm_quant   h = bf16(x + residual), y = bf16(h / rms(h) * weight), y as
                   int8 or E4M3 codes with a scale per group
  rms_norm_bwd     the gradients of that norm for h (x and residual share it)
                   and for the weight
  mxfp4_quant      bf16 rows as E2M1 codes with an E8M0 scale per 32 values,
                   along the rows and, for training, along the columns too
  mxfp4_gemm       C = A . B^T of two such operands
  group_dequant, mxfp4_dequant   the values that codes and scales stand for

Codes are returned as the values they stand for, in bf16, through the
dequantiser, so a pass that quantises holds both.
"""

import math

import torch

own = False

EPS = 1e-6
MAX_PAIRS = 16384 * 4096           # elements of a drawn norm or quantiser case
MAX_PRODUCTS = 16384 * 22016 * 4096  # M * N * K of a drawn product


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # one new token of a served model: launch latency
        dict(name="norm_t1", op="norm", T=1, D=4096, codes="int8", group=128, residual=True, x="bf16"),
        # a training batch ahead of the int8 gate/up product
        dict(name="norm_t16384", op="norm", T=16384, D=4096, codes="int8", group=128, residual=True, x="bf16"),
        # ragged rows: an odd width, a short last group, E4M3 codes, the fp32 output of a product as x
        dict(name="norm_t999_d1001_e4m3", op="norm", T=999, D=1001, codes="e4m3", group=64, residual=True, x="f32"),
        # the same training batch's backward: gradient from the dgrad product in bf16, joined by the residual's own
        dict(name="norm_bwd_t16384", op="norm_bwd", T=16384, D=4096, dy="bf16", d_h=True),
        # a short micro-batch of an odd width, the gradient in fp32
        dict(name="norm_bwd_t333_d2050", op="norm_bwd", T=333, D=2050, dy="f32", d_h=True),
        # activations of a few served sequences on their way into a 4-bit product
        dict(name="quant_r8_k11008", op="quant", R=8, K=11008, both=False),
        # a training batch along both axes: rows for the forward product, columns for the weight's gradient
        dict(name="quant_both_r8192_k4096", op="quant", R=8192, K=4096, both=True),
        # one token through the gate/up weight: the weight is read once, nothing else counts
        dict(name="gemm_m1", op="gemm", M=1, N=22016, K=4096, out="bf16"),
        # a batch of served sequences through the down weight
        dict(name="gemm_m64", op="gemm", M=64, N=4096, K=11008, out="bf16"),
        # ragged everywhere: a prompt of 777 tokens, a width off every tile, K off the 128 wide steps
        dict(name="gemm_m777_n1001_k1376", op="gemm", M=777, N=1001, K=1376, out="f32"),
        # the gate/up product of a training batch
        dict(name="gemm_m16384", op="gemm", M=16384, N=22016, K=4096, out="bf16"),
        # a 4-bit weight back in bf16, for a consumer without a 4-bit product
        dict(name="dequant_n22016_k4096", op="dequant", R=22016, K=4096, codes="mxfp4", group=32),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(("norm", "norm", "norm_bwd", "norm_bwd", "quant", "quant", "gemm", "gemm", "gemm", "gemm", "dequant"))
    if op == "gemm":
        M = _log_int(rng, 1, 16384)
        N = _log_int(rng, 1, 22016)
        K = 32 * _log_int(rng, 1, min(22016, MAX_PRODUCTS // (M * N)) // 32)
        return dict(op=op, M=M, N=N, K=K, out=rng.choice(("f32", "bf16")))
    rows = _log_int(rng, 1, 32768)
    cols = _log_int(rng, 1, min(16384, MAX_PAIRS // rows))
    if rng.random() < 0.5 and cols >= 64:
        cols -= cols % 32  # half of the widths are whole blocks, the others whatever they are
    if op == "norm":
        return dict(op=op, T=rows, D=cols, codes=rng.choice(("int8", "e4m3")), group=rng.choice((32, 64, 128)),
                    residual=rng.random() < 0.7, x=rng.choice(("bf16", "f32")))
    if op == "norm_bwd":
        return dict(op=op, T=rows, D=cols, dy=rng.choice(("bf16", "f32")), d_h=rng.random() < 0.7)
    if op == "quant":
        return dict(op=op, R=rows, K=cols, both=rng.random() < 0.5)
    codes = rng.choice(("int8", "e4m3", "mxfp4"))
    return dict(op=op, R=rows, K=cols, codes=codes, group=32 if codes == "mxfp4" else rng.choice((32, 64, 128)))


def _blocks(n, group=32):
    return -(-n // group)


def work(case):
    c = case
    if c["op"] == "norm":
        n, x = c["T"] * c["D"], 4 if c["x"] == "f32" else 2
        scales = 4 * c["T"] * _blocks(c["D"], c["group"])
        # x, residual, weight in; h, codes, scales, rstd and the codes' values out
        return {"bytes": n * (x + (2 if c["residual"] else 0) + 2 + 1 + 2) + scales + 4 * c["T"] + 2 * c["D"], "flops": 8 * n}
    if c["op"] == "norm_bwd":
        n, dy = c["T"] * c["D"], 4 if c["dy"] == "f32" else 2
        return {"bytes": n * (dy + 2 + (2 if c["d_h"] else 0) + 2) + 4 * c["T"] + 6 * c["D"], "flops": 9 * n}
    if c["op"] == "quant":
        n = c["R"] * c["K"]
        rows = 17 * c["R"] * _blocks(c["K"]) + 2 * n      # codes and scales, and their values
        cols = 17 * c["K"] * _blocks(c["R"]) + 2 * n
        return {"bytes": 2 * n + rows + (cols if c["both"] else 0), "flops": 4 * n * (2 if c["both"] else 1)}
    if c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": (M + N) * (K // 2 + K // 32) + M * N * (4 if c["out"] == "f32" else 2), "flops": 2 * M * N * K}
    n = c["R"] * c["K"]
    codes = 17 * c["R"] * _blocks(c["K"]) if c["codes"] == "mxfp4" else n + 4 * c["R"] * _blocks(c["K"], c["group"])
    return {"bytes": codes + 2 * n, "flops": n}


# ---- the formats, plainly ---------------------------------------------------

def _grouped(v, group):
    """[R, K] as [R, groups, group], the last group filled up with zeros."""
    fill = -v.shape[1] % group
    return torch.nn.functional.pad(v, (0, fill)).view(v.shape[0], -1, group)


def _group_quant(y, codes, group):
    """Codes (as fp32 numbers) and scales of the fp32 rows y, by group: scale =
    amax / 127 or / 448 (1 for a group of zeros), code = the nearest to y * (1 / scale)."""
    g = _grouped(y, group)
    amax = g.abs().amax(2, keepdim=True)
    scale = torch.where(amax == 0, torch.ones_like(amax), amax / (448.0 if codes == "e4m3" else 127.0))
    p = g * (1.0 / scale)
    if codes == "e4m3":
        q = p.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()
    else:
        q = torch.round(p).clamp(-127.0, 127.0)
    return q, scale


def _mx_quant(x):
    """E2M1 magnitudes with signs (as fp32 numbers, [R, blocks, 32]) and E8M0
    exponents [R, blocks, 1] of the fp32 rows x: the exponent of a block is
    floor(log2(amax)) - 2, at least -127; 0 for a block of zeros."""
    g = _grouped(x, 32)
    amax = g.abs().amax(2, keepdim=True)
    e = (torch.frexp(amax)[1] - 3).clamp(min=-127)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    v = g * torch.exp2(-e.float())
    a = v.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    return torch.copysign((torch.round(a / step) * step).clamp(max=6.0), v), e


def _mx_pack(q, e):
    """The stored form: two codes to a byte (the even one in the low half), a byte per exponent."""
    levels = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=q.device)
    code = torch.bucketize(q.abs(), levels) + 8 * torch.signbit(q)
    code = code.view(q.shape[0], -1).to(torch.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), (e[..., 0] + 127).to(torch.uint8)


def _mx_values(q, s):
    """The fp32 numbers that packed codes q [R, 16 * blocks] and exponents s [R, blocks] stand for."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
    table = torch.cat([table, -table])
    code = torch.stack([q & 15, q >> 4], 2).view(q.shape[0], -1, 32)
    return (table[code.int()] * torch.exp2(s.float() - 127.0)[..., None]).view(q.shape[0], -1)


# ---- inputs -----------------------------------------------------------------

def _normal(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda") * std


def _stream(g, rows, cols):
    """Rows of a residual stream: a scale per row, a few loud channels, and a row of zeros (padding) in 97."""
    v = _normal(g, rows, cols) * torch.exp(_normal(g, rows, 1, std=0.5))
    v *= torch.where(torch.rand(cols, generator=g, device="cuda") < 0.005, 20.0, 1.0)
    v[96::97] = 0
    return v


def _weight(g, n):
    return (1.0 + _normal(g, n, std=0.2)).to(torch.bfloat16)


def _code_type(codes):
    return torch.int8 if codes == "int8" else torch.float8_e4m3fn


def _buffer(*shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    bf16, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    state = {"case": dict(c)}
    if c["op"] == "norm":
        T, D = c["T"], c["D"]
        state["x"] = _stream(g, T, D).to(f32 if c["x"] == "f32" else bf16)
        state["residual"] = _stream(g, T, D).to(bf16) if c["residual"] else None
        state["weight"] = _weight(g, D)
        state["q"] = _buffer(T, D, dtype=_code_type(c["codes"]))
        state["s"] = _buffer(T, _blocks(D, c["group"]), dtype=f32)
        state["h"], state["rstd"] = _buffer(T, D, dtype=bf16), _buffer(T, dtype=f32)
        state["values"] = _buffer(T, D, dtype=bf16)
    elif c["op"] == "norm_bwd":
        T, D = c["T"], c["D"]
        h = (_normal(g, T, D) * torch.exp(_normal(g, T, 1, std=0.5))).to(bf16)
        state["h"], state["weight"] = h, _weight(g, D)
        state["rstd"] = 1.0 / torch.sqrt((h.float() * h.float()).mean(1) + EPS)
        state["dy"] = _normal(g, T, D, std=0.01).to(f32 if c["dy"] == "f32" else bf16)
        state["d_h"] = _normal(g, T, D, std=0.01).to(bf16) if c["d_h"] else None
        state["dx"], state["dw"] = _buffer(T, D, dtype=bf16), _buffer(D, dtype=f32)
    elif c["op"] == "quant":
        R, K = c["R"], c["K"]
        state["x"] = _stream(g, R, K).to(bf16)
        state["q"], state["s"] = _buffer(R, 16 * _blocks(K), dtype=u8), _buffer(R, _blocks(K), dtype=u8)
        state["values"] = _buffer(R, K, dtype=bf16)
        if c["both"]:
            state["q_t"], state["s_t"] = _buffer(K, 16 * _blocks(R), dtype=u8), _buffer(K, _blocks(R), dtype=u8)
            state["values_t"] = _buffer(K, R, dtype=bf16)
    elif c["op"] == "gemm":
        M, N, K = c["M"], c["N"], c["K"]
        state["A"], state["sA"] = _mx_pack(*_mx_quant(_stream(g, M, K)))
        state["B"], state["sB"] = _mx_pack(*_mx_quant(_normal(g, N, K, std=0.02)))
        state["C"] = _buffer(M, N, dtype=f32 if c["out"] == "f32" else bf16)
    else:
        v = _stream(g, c["R"], c["K"])
        if c["codes"] == "mxfp4":
            state["q"], state["s"] = _mx_pack(*_mx_quant(v))
        else:
            q, s = _group_quant(v, c["codes"], c["group"])
            state["q"] = q.view(c["R"], -1)[:, :c["K"]].to(_code_type(c["codes"])).contiguous()
            state["s"] = s[..., 0].contiguous()
        state["values"] = _buffer(c["R"], c["K"], dtype=bf16)
    return state


# ---- one pass ---------------------------------------------------------------

def run(state):
    return _run_library(state) if own else _run_plain(state)


def _run_plain(state):
    c = state["case"]
    bf16 = torch.bfloat16
    if c["op"] == "norm":
        h = state["x"].float()
        if state["residual"] is not None:
            h = h + state["residual"].float()
        h = h.to(bf16)
        v = h.float()
        rstd = 1.0 / torch.sqrt((v * v).sum(1) / c["D"] + EPS)
        y = ((v * rstd[:, None]) * state["weight"].float()).to(bf16)
        q, s = _group_quant(y.float(), c["codes"], c["group"])
        return {"h": h, "rstd": rstd, "y": (q * s).view(c["T"], -1)[:, :c["D"]].to(bf16)}
    if c["op"] == "norm_bwd":
        n = state["h"].float() * state["rstd"][:, None]
        dy = state["dy"].float()
        g = dy * state["weight"].float()
        dx = state["rstd"][:, None] * (g - n * ((g * n).sum(1, keepdim=True) / c["D"]))
        if state["d_h"] is not None:
            dx = dx + state["d_h"].float()
        return {"dx": dx.to(bf16), "dw": (dy * n).sum(0)}
    if c["op"] == "quant":
        x = state["x"].float()
        q, e = _mx_quant(x)
        out = {"values": (q * torch.exp2(e.float())).view(c["R"], -1)[:, :c["K"]].to(bf16)}
        if c["both"]:
            q, e = _mx_quant(x.t())
            out["values_t"] = (q * torch.exp2(e.float())).view(c["K"], -1)[:, :c["R"]].to(bf16)
        return out
    if c["op"] == "gemm":
        C = _mx_values(state["A"], state["sA"]) @ _mx_values(state["B"], state["sB"]).t()
        return {"C": C if c["out"] == "f32" else C.to(bf16)}
    if c["codes"] == "mxfp4":
        v = _mx_values(state["q"], state["s"])
    else:
        v = (_grouped(state["q"].float(), c["group"]) * state["s"][..., None]).view(c["R"], -1)
    return {"values": v[:, :c["K"]].to(bf16)}


def _run_library(state):
    import swiglu_backward_int8_amd as sq

    c = state["case"]
    if c["op"] == "norm":
        sq.rms_norm_quant(state["x"], state["weight"], state["q"], state["s"], residual=state["residual"], h=state["h"],
                          rstd=state["rstd"], eps=EPS, group_size=c["group"])
        sq.group_dequant(state["q"], state["s"], state["values"], group_size=c["group"])
        return {"h": state["h"], "rstd": state["rstd"], "y": state["values"]}
    if c["op"] == "norm_bwd":
        if "workspace" not in state:  # kept, as a training loop keeps it
            state["workspace"] = sq.rms_norm_bwd_workspace(c["T"], c["D"], state["h"].device)
        sq.rms_norm_bwd(state["dy"], state["h"], state["weight"], state["rstd"], state["dx"], dw=state["dw"],
                        d_h=state["d_h"], workspace=state["workspace"])
        return {"dx": state["dx"], "dw": state["dw"]}
    if c["op"] == "quant":
        out = {"values": state["values"]}
        if c["both"]:
            sq.mxfp4_quant(state["x"], state["q"], state["s"], q_t=state["q_t"], s_t=state["s_t"])
            sq.mxfp4_dequant(state["q_t"], state["s_t"], state["values_t"])
            out["values_t"] = state["values_t"]
        else:
            sq.mxfp4_quant(state["x"], state["q"], state["s"])
        sq.mxfp4_dequant(state["q"], state["s"], state["values"])
        return out
    if c["op"] == "gemm":
        sq.mxfp4_gemm(state["A"], state["sA"], state["B"], state["sB"], state["C"])
        return {"C": state["C"]}
    if c["codes"] == "mxfp4":
        sq.mxfp4_dequant(state["q"], state["s"], state["values"])
    else:
        sq.group_dequant(state["q"], state["s"], state["values"], group_size=c["group"])
    return {"values": state["values"]}


# ---- the definitions in 64 bits ---------------------------------------------

def _nearest(v, levels):
    """v rounded to the nearest of the sorted levels (a tie goes to the level of even index), beyond them to the last."""
    mid = (levels[1:] + levels[:-1]) / 2
    a = v.abs().contiguous()
    low, high = torch.bucketize(a, mid), torch.bucketize(a, mid, right=True)  # they differ at a tie alone
    return torch.where(v < 0, -1.0, 1.0) * levels[torch.where(low % 2 == 0, low, high)]


def _segments(v, size):
    """The columns of v in runs of `size`, the short last run filled up with zeros."""
    runs = -(-v.shape[1] // size)
    wide = torch.zeros((v.shape[0], runs * size), dtype=torch.float64, device=v.device)
    wide[:, :v.shape[1]] = v
    return wide.reshape(v.shape[0], runs, size)


def _exact_mx(x):
    levels = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    b = _segments(x.double(), 32)
    top = b.abs().max(2, keepdim=True).values
    scale = torch.exp2(torch.floor(torch.log2(torch.where(top > 0, top, 4.0))) - 2).clamp(min=2.0**-127)
    return (_nearest(b / scale, levels) * scale).reshape(x.shape[0], -1)[:, :x.shape[1]]


def _exact_decode(q, s):
    """Packed E2M1 codes: sign, two exponent bits, one fraction bit; exponents with bias 127."""
    c = torch.empty((q.shape[0], 2 * q.shape[1]), dtype=torch.int64, device=q.device)
    c[:, 0::2], c[:, 1::2] = (q & 15).long(), (q >> 4).long()
    e, f = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e == 0, 0.5 * f, (1 + 0.5 * f) * torch.exp2(e.double() - 1))
    v = torch.where(c >= 8, -v, v).reshape(q.shape[0], -1, 32)
    return torch.ldexp(v, (s.long() - 127)[..., None]).reshape(q.shape[0], -1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            h = h + s["residual"].double()
        h = h.to(torch.bfloat16).double()  # rounded by definition: what the residual stream holds
        rstd = (h.square().mean(1) + EPS) ** -0.5
        y = (h * rstd[:, None] * s["weight"].double()).to(torch.bfloat16).double()  # so is what is quantised
        b = _segments(y, c["group"])
        top = b.abs().max(2, keepdim=True).values
        if c["codes"] == "int8":
            v = torch.round(b / torch.where(top > 0, top, 1.0) * 127.0) * top / 127.0
        else:
            m = torch.arange(8, dtype=torch.float64, device=b.device) / 8
            p = torch.exp2(torch.arange(-6, 9, dtype=torch.float64, device=b.device))
            levels = torch.cat([m * 2.0**-6, ((1 + m) * p[:, None]).reshape(-1)])[:-1]  # 0 to 448: the last pattern is NaN
            v = _nearest(b / torch.where(top > 0, top, 1.0) * 448.0, levels) * top / 448.0
        return {"h": h, "rstd": rstd, "y": v.reshape(c["T"], -1)[:, :c["D"]]}
    if c["op"] == "norm_bwd":
        n = s["h"].double() * s["rstd"].double()[:, None]
        w, dy = s["weight"].double(), s["dy"].double()
        dx = s["rstd"].double()[:, None] * (dy * w - n * (dy * w * n).mean(1, keepdim=True))
        return {"dx": dx + s["d_h"].double() if s["d_h"] is not None else dx, "dw": (dy * n).sum(0)}
    if c["op"] == "quant":
        out = {"values": _exact_mx(s["x"])}
        if c["both"]:
            out["values_t"] = _exact_mx(s["x"].t().contiguous())
        return out
    if c["op"] == "gemm":
        return {"C": _exact_decode(s["A"], s["sA"]) @ _exact_decode(s["B"], s["sB"]).t()}
    if c["codes"] == "mxfp4":
        return {"values": _exact_decode(s["q"], s["s"])[:, :c["K"]]}
    v = _segments(s["q"].double(), c["group"]) * s["s"].double()[..., None]
    return {"values": v.reshape(c["R"], -1)[:, :c["K"]]}
