"""The layer norm, dropout and gated projection as they are measured: cases,
inputs, the plain form of each operator in elementary torch operations, the
library's calls, and the operators' definitions in 64 bits.

  layer_norm_quant  h = bf16(residual + dropout(x)), y = bf16((h - mean) * rstd *
                    weight + bias), y as bf16 or as int8 or E4M3 codes with a
                    scale per group
  layer_norm_bwd    the gradients of that norm for h, for x (through the dropout),
                    for the weight and for the bias
  dropout_add       residual + dropout(x): the forward pass; without a residual,
                    on the gradient, the backward pass
  swiglu_gemm       y = silu(x Wg^T) * (x Wu^T) in one kernel, W = [Wg; Wu]
  swiglu_gemm_bwd   the gradients of that for [gate | up], x and W

The mask of a dropout is a function of the place and of rng, two 64-bit numbers:
Philox4x32 with ten rounds (Salmon, Moraes, Dror and Shaw, "Parallel random
numbers: as easy as 1, 2, 3", 2011), key rng[0], counter (column / 4, row, rng[1]);
word column % 4 decides, and below p * 2^32 the element is dropped.  Codes are
returned as the values they stand for, in bf16, through the dequantiser.
"""

import math

import torch

own = False

EPS = 1e-5
MAX_PAIRS = 16384 * 4096               # elements of a drawn norm case
MAX_DROPPED = 16384 * 11008            # elements of a drawn dropout case
MAX_PRODUCTS = 16384 * 11008 * 4096    # T * H * D of a drawn projection


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # one new token of a served model, int8 codes for the next product: launch latency
        dict(name="norm_t1", op="norm", T=1, D=4096, out="int8", group=128, residual=True, x="bf16", p=0.0),
        # a training batch: the sub-layer's output dropped out and added to the stream, y for a bf16 product
        dict(name="norm_t16384_p10", op="norm", T=16384, D=4096, out="bf16", group=128, residual=True, x="bf16", p=0.1),
        # ragged rows: an odd width, a short last group, E4M3 codes, the fp32 output of a product as x
        dict(name="norm_t999_d1001_e4m3", op="norm", T=999, D=1001, out="e4m3", group=64, residual=True, x="f32", p=0.0),
        # the training batch's backward: both streams' gradients and both parameters'
        dict(name="norm_bwd_t16384_p10", op="norm_bwd", T=16384, D=4096, dy="bf16", d_h=True, p=0.1),
        # a short micro-batch of an odd width, the gradient in fp32
        dict(name="norm_bwd_t333_d2050", op="norm_bwd", T=333, D=2050, dy="f32", d_h=False, p=0.0),
        # a fine-tuning micro-batch on its way into the residual stream
        dict(name="dropout_t256_d4096", op="dropout", T=256, D=4096, residual=True, x="bf16", p=0.1),
        # the activations between the two projections of a training batch (or their gradient)
        dict(name="dropout_t16384_d11008", op="dropout", T=16384, D=11008, residual=False, x="bf16", p=0.25),
        # one token through the gate and up projections: the weight is read once, nothing else counts
        dict(name="swiglu_t1", op="swiglu", T=1, H=11008, D=4096, gu=False),
        # a prompt of a few hundred tokens through a small block, off every tile; gate and up kept
        dict(name="swiglu_t777_h1376_d2048", op="swiglu", T=777, H=1376, D=2048, gu=True),
        # a training batch: gate and up kept for the backward pass
        dict(name="swiglu_t16384", op="swiglu", T=16384, H=11008, D=4096, gu=True),
        # its backward pass
        dict(name="swiglu_bwd_t16384", op="swiglu_bwd", T=16384, H=11008, D=4096),
        # the backward pass of a micro-batch off every tile
        dict(name="swiglu_bwd_t1001_h1408_d1032", op="swiglu_bwd", T=1001, H=1408, D=1032),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(("norm", "norm", "norm_bwd", "norm_bwd", "dropout", "swiglu", "swiglu", "swiglu_bwd", "swiglu_bwd"))
    if op in ("swiglu", "swiglu_bwd"):
        T = _log_int(rng, 1 if op == "swiglu" else 16, 16384)
        H = 8 * _log_int(rng, 8, 11008 // 8)
        D = 8 * _log_int(rng, 8, min(8192, MAX_PRODUCTS // (T * H)) // 8)
        return dict(op=op, T=T, H=H, D=D, gu=rng.random() < 0.5) if op == "swiglu" else dict(op=op, T=T, H=H, D=D)
    rows = _log_int(rng, 1, 32768)
    cols = _log_int(rng, 1, min(16384, (MAX_DROPPED if op == "dropout" else MAX_PAIRS) // rows))
    if rng.random() < 0.5 and cols >= 64:
        cols -= cols % 32  # half of the widths are whole blocks, the others whatever they are
    p = rng.choice((0.0, 0.05, 0.1, 0.3))
    if op == "norm":
        return dict(op=op, T=rows, D=cols, out=rng.choice(("bf16", "int8", "e4m3")), group=rng.choice((32, 64, 128)),
                    residual=rng.random() < 0.7, x=rng.choice(("bf16", "f32")), p=p)
    if op == "norm_bwd":
        return dict(op=op, T=rows, D=cols, dy=rng.choice(("bf16", "f32")), d_h=rng.random() < 0.7, p=p)
    return dict(op=op, T=rows, D=cols, residual=rng.random() < 0.5, x=rng.choice(("bf16", "f32")), p=p or 0.5)


def work(case):
    c = case
    T = c["T"]
    if c["op"] in ("swiglu", "swiglu_bwd"):
        H, D = c["H"], c["D"]
        if c["op"] == "swiglu":  # x, W in; y and perhaps gate and up out
            return {"bytes": 2 * T * D + 4 * H * D + (6 if c["gu"] else 2) * T * H, "flops": 4 * T * H * D}
        # dy, gate and up, x, W in; the gradients of gate and up, x, W out
        return {"bytes": 10 * T * H + 4 * T * D + 8 * H * D, "flops": 8 * T * H * D}
    n = T * c["D"]
    x = 4 if c.get("x", c.get("dy")) == "f32" else 2
    mask = 20 * n if c["p"] > 0 else 0  # two 32-bit products in each of ten rounds for four elements, and as many sums
    if c["op"] == "norm":
        y = 2 if c["out"] == "bf16" else 3  # codes and their values
        scales = 0 if c["out"] == "bf16" else 4 * T * -(-c["D"] // c["group"])
        return {"bytes": n * (x + (2 if c["residual"] else 0) + 2 + y) + scales + 8 * T, "flops": 12 * n + mask}
    if c["op"] == "norm_bwd":
        return {"bytes": n * (x + 2 + (2 if c["d_h"] else 0) + 2 + (2 if c["p"] > 0 else 0)) + 8 * T, "flops": 14 * n + mask}
    return {"bytes": n * (x + (2 if c["residual"] else 0) + 2), "flops": 2 * n + mask}


# ---- the formats, plainly ---------------------------------------------------

M32 = 0xFFFFFFFF


def _mask(rng, T, D, p):
    """Which elements of a [T, D] tensor a dropout keeps."""
    dev = rng.device
    # 64-bit integers: a product of two 32-bit words keeps its bits, whatever its sign
    seed, step = rng[0], rng[1]
    k0, k1 = seed & M32, (seed >> 32) & M32
    shape = (T, -(-D // 4))
    c0 = torch.arange(shape[1], dtype=torch.int64, device=dev).expand(shape)
    c1 = torch.arange(T, dtype=torch.int64, device=dev)[:, None].expand(shape)
    c2, c3 = (step & M32).expand(shape), ((step >> 32) & M32).expand(shape)
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & M32) ^ c1 ^ k0, b & M32, ((a >> 32) & M32) ^ c3 ^ k1, a & M32
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    words = torch.stack((c0, c1, c2, c3), 2).view(T, -1)[:, :D]
    return words >= round(_f32(p) * 2**32)


def _f32(p):
    return float(torch.tensor(p, dtype=torch.float32))


def _scale(p):
    """What kept elements are multiplied by: one fp32 number."""
    return _f32(1.0 / (1.0 - _f32(p)))


def _dropped(v, rng, p):
    """fp32 rows v through a dropout."""
    if p == 0:
        return v
    return torch.where(_mask(rng, *v.shape, p), v * _scale(p), torch.zeros_like(v))


def _grouped(v, group):
    """[R, K] as [R, groups, group], the last group filled up with zeros."""
    return torch.nn.functional.pad(v, (0, -v.shape[1] % group)).view(v.shape[0], -1, group)


def _group_values(y, codes, group):
    """The bf16 values of the codes of the fp32 rows y: scale = amax / 127 or / 448
    by group (1 for a group of zeros), code = the nearest to y * (1 / scale)."""
    g = _grouped(y, group)
    amax = g.abs().amax(2, keepdim=True)
    scale = torch.where(amax == 0, torch.ones_like(amax), amax / (448.0 if codes == "e4m3" else 127.0))
    q = g * (1.0 / scale)
    if codes == "e4m3":
        q = q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()
    else:
        q = torch.round(q).clamp(-127.0, 127.0)
    return (q * scale).view(y.shape[0], -1)[:, :y.shape[1]].to(torch.bfloat16)


# ---- inputs -----------------------------------------------------------------

def _normal(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda") * std


def _stream(g, rows, cols):
    """Rows of a residual stream: a scale and an offset per row, a few loud channels, a row of zeros (padding) in 97."""
    v = _normal(g, rows, cols) * torch.exp(_normal(g, rows, 1, std=0.5))
    v *= torch.where(torch.rand(cols, generator=g, device="cuda") < 0.005, 20.0, 1.0)
    v += 0.3 + _normal(g, rows, 1, std=0.1)
    v[96::97] = 0
    return v


def _buffer(*shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    bf16, f32 = torch.bfloat16, torch.float32
    T = c["T"]
    state = {"case": dict(c)}
    if c["op"] in ("swiglu", "swiglu_bwd"):
        H, D = c["H"], c["D"]
        state["x"] = (_normal(g, T, D) * torch.exp(_normal(g, D, std=0.3))).to(bf16)  # a norm's output
        state["w"] = _normal(g, 2 * H, D, std=D**-0.5).to(bf16)
        if c["op"] == "swiglu":
            state["y"] = _buffer(T, H, dtype=bf16)
            state["gu"] = _buffer(T, 2 * H, dtype=bf16) if c["gu"] else None
        else:
            state["gu"] = _normal(g, T, 2 * H).to(bf16)
            state["dy"] = _normal(g, T, H, std=0.01).to(bf16)
            state["d_gu"] = _buffer(T, 2 * H, dtype=bf16)
            state["dx"], state["dw"] = _buffer(T, D, dtype=bf16), _buffer(2 * H, D, dtype=bf16)
        return state
    D = c["D"]
    state["rng"] = torch.randint(-2**62, 2**62, (2,), generator=g, device="cuda")  # the seed and the step's number
    if c["op"] == "dropout":
        state["x"] = _normal(g, T, D).to(f32 if c["x"] == "f32" else bf16)
        state["residual"] = _stream(g, T, D).to(bf16) if c["residual"] else None
        state["out"] = _buffer(T, D, dtype=bf16)
        return state
    state["weight"] = (1.0 + _normal(g, D, std=0.2)).to(bf16)
    state["h"] = _buffer(T, D, dtype=bf16)
    if c["op"] == "norm":
        state["bias"] = _normal(g, D, std=0.1).to(bf16)
        state["x"] = _stream(g, T, D).to(f32 if c["x"] == "f32" else bf16)
        state["residual"] = _stream(g, T, D).to(bf16) if c["residual"] else None
        state["mean"], state["rstd"], state["y"] = (_buffer(T, dtype=f32), _buffer(T, dtype=f32), _buffer(T, D, dtype=bf16))
        if c["out"] != "bf16":
            state["q"] = _buffer(T, D, dtype=torch.int8 if c["out"] == "int8" else torch.float8_e4m3fn)
            state["s"] = _buffer(T, -(-D // c["group"]), dtype=f32)
    else:
        h = _stream(g, T, D).to(bf16)
        state["h"] = h
        state["mean"] = h.float().mean(1)
        state["rstd"] = 1.0 / torch.sqrt((h.float() - state["mean"][:, None]).square().mean(1) + EPS)
        state["dy"] = _normal(g, T, D, std=0.01).to(f32 if c["dy"] == "f32" else bf16)
        state["d_h"] = _normal(g, T, D, std=0.01).to(bf16) if c["d_h"] else None
        state["dx"] = _buffer(T, D, dtype=bf16)
        state["dx_drop"] = _buffer(T, D, dtype=bf16) if c["p"] > 0 else None
        state["dw"], state["db"] = _buffer(D, dtype=f32), _buffer(D, dtype=f32)
    return state


# ---- one pass ---------------------------------------------------------------

def run(state):
    return _run_library(state) if own else _run_plain(state)


def _run_plain(state):
    c = state["case"]
    bf16 = torch.bfloat16
    if c["op"] == "norm":
        v = _dropped(state["x"].float(), state["rng"], c["p"])
        if state["residual"] is not None:
            v = v + state["residual"].float()
        h = v.to(bf16)  # rounded by definition: what the residual stream holds
        v = h.float()
        mean = v.sum(1) / c["D"]
        v = v - mean[:, None]
        rstd = 1.0 / torch.sqrt((v * v).sum(1) / c["D"] + EPS)
        y = ((v * rstd[:, None]) * state["weight"].float() + state["bias"].float()).to(bf16)
        if c["out"] != "bf16":
            y = _group_values(y.float(), c["out"], c["group"])
        return {"h": h, "mean": mean, "rstd": rstd, "y": y}
    if c["op"] == "norm_bwd":
        n = (state["h"].float() - state["mean"][:, None]) * state["rstd"][:, None]
        dy = state["dy"].float()
        g = dy * state["weight"].float()
        dx = state["rstd"][:, None] * (g - g.sum(1, keepdim=True) / c["D"] - n * ((g * n).sum(1, keepdim=True) / c["D"]))
        if state["d_h"] is not None:
            dx = dx + state["d_h"].float()
        out = {"dx": dx.to(bf16), "dw": (dy * n).sum(0), "db": dy.sum(0)}
        if c["p"] > 0:
            out["dx_drop"] = _dropped(dx, state["rng"], c["p"]).to(bf16)
        return out
    if c["op"] == "dropout":
        v = _dropped(state["x"].float(), state["rng"], c["p"])
        return {"out": (v + state["residual"].float() if state["residual"] is not None else v).to(bf16)}
    if c["op"] == "swiglu":
        gate, up = (state["x"].float() @ state["w"].float().t()).chunk(2, 1)
        out = {"y": (gate / (1.0 + torch.exp(-gate)) * up).to(bf16)}
        if c["gu"]:
            out["gu"] = torch.cat([gate, up], 1).to(bf16)
        return out
    gate, up = state["gu"].float().chunk(2, 1)
    dy = state["dy"].float()
    s = 1.0 / (1.0 + torch.exp(-gate))
    d_gu = torch.cat([dy * up * s * (1.0 + gate * (1.0 - s)), dy * (gate * s)], 1).to(bf16)  # rounded by definition
    d = d_gu.float()
    return {"d_gu": d_gu, "dx": (d @ state["w"].float()).to(bf16), "dw": (d.t() @ state["x"].float()).to(bf16)}


def _run_library(state):
    import swiglu_backward_int8_amd as sq

    c = state["case"]
    if c["op"] == "norm":
        coded = c["out"] != "bf16"
        sq.layer_norm_quant(state["x"], state["weight"], bias=state["bias"], y_q=state["q"] if coded else None,
                            y_s=state["s"] if coded else None, residual=state["residual"], h=state["h"],
                            mean=state["mean"], rstd=state["rstd"], y_bf16=None if coded else state["y"], eps=EPS,
                            group_size=c["group"], p=c["p"], rng=state["rng"] if c["p"] > 0 else None)
        if coded:
            sq.group_dequant(state["q"], state["s"], state["y"], group_size=c["group"])
        return {"h": state["h"], "mean": state["mean"], "rstd": state["rstd"], "y": state["y"]}
    if c["op"] == "norm_bwd":
        if "workspace" not in state:  # kept, as a training loop keeps it
            state["workspace"] = sq.layer_norm_bwd_workspace(c["T"], c["D"], state["h"].device)
        sq.layer_norm_bwd(state["dy"], state["h"], state["weight"], state["mean"], state["rstd"], state["dx"],
                          dw=state["dw"], db=state["db"], d_h=state["d_h"], dx_drop=state["dx_drop"],
                          workspace=state["workspace"], p=c["p"], rng=state["rng"] if c["p"] > 0 else None)
        out = {"dx": state["dx"], "dw": state["dw"], "db": state["db"]}
        if c["p"] > 0:
            out["dx_drop"] = state["dx_drop"]
        return out
    if c["op"] == "dropout":
        sq.dropout_add(state["x"], state["out"], c["p"], state["rng"], residual=state["residual"])
        return {"out": state["out"]}
    if c["op"] == "swiglu":
        sq.swiglu_gemm(state["x"], state["w"], state["y"], gu=state["gu"])
        return {"y": state["y"], "gu": state["gu"]} if c["gu"] else {"y": state["y"]}
    if "workspace" not in state:
        state["workspace"] = sq.swiglu_gemm_bwd_workspace(c["T"], c["H"], c["D"], state["x"].device)
    sq.swiglu_gemm_bwd(state["dy"], state["gu"], state["x"], state["w"], state["d_gu"], dx=state["dx"], dw=state["dw"],
                       workspace=state["workspace"])
    return {"d_gu": state["d_gu"], "dx": state["dx"], "dw": state["dw"]}


# ---- the definitions in 64 bits ---------------------------------------------

def _philox_words(key, counter):
    """The four words of one block, ten rounds; everything in halves of 16 bits, so that nothing passes 63 bits."""
    def product(c, m):
        lo, hi = (c & 0xFFFF) * m, (c >> 16) * m
        low = lo + ((hi & 0xFFFF) << 16)
        return (hi >> 16) + (low >> 32), low & M32

    c, (k0, k1) = list(counter), key
    for r in range(10):
        h0, l0 = product(c[0], 0xD2511F53)
        h1, l1 = product(c[2], 0xCD9E8D57)
        c = [h1 ^ c[1] ^ ((k0 + r * 0x9E3779B9) % 2**32), l1, h0 ^ c[3] ^ ((k1 + r * 0xBB67AE85) % 2**32), l0]
    return c


def _exact_dropped(v, rng, p):
    if p == 0:
        return v
    seed, step = (int(t) % 2**64 for t in rng.tolist())
    T, D = v.shape
    col = torch.arange(-(-D // 4), device=v.device)[None, :]
    row = torch.arange(T, device=v.device)[:, None]
    zero = torch.zeros_like(row + col)
    words = _philox_words((seed % 2**32, seed >> 32), (zero + col, zero + row, zero + step % 2**32, zero + (step >> 32)))
    p = _f32(p)
    out = torch.zeros_like(v)
    for j, word in enumerate(words):
        part = v[:, j::4]
        kept = word[:, :part.shape[1]].double() >= p * 2.0**32
        out[:, j::4] = torch.where(kept, part * _scale(p), 0.0)
    return out


def _exact_stream(s, p):
    """residual + dropout(x): by definition one fp32 product and one fp32 sum.  With a scale such as 10 / 9 one
    value in a few hundred is within 1e-7 of halfway between two bf16 numbers."""
    v = _exact_dropped(s["x"].double(), s["rng"], p).float().double()
    return v if s["residual"] is None else (v + s["residual"].double()).float().double()


def _segments(v, size):
    """The columns of v in runs of `size`, the short last run filled up with zeros."""
    runs = -(-v.shape[1] // size)
    wide = torch.zeros((v.shape[0], runs * size), dtype=torch.float64, device=v.device)
    wide[:, :v.shape[1]] = v
    return wide.reshape(v.shape[0], runs, size)


def _exact_codes(y, codes, group):
    b = _segments(y, group)
    top = b.abs().max(2, keepdim=True).values
    unit = b / torch.where(top > 0, top, 1.0)
    if codes == "int8":
        v = torch.round(unit * 127.0) * top / 127.0
    else:
        m = torch.arange(8, dtype=torch.float64, device=b.device) / 8
        e = torch.exp2(torch.arange(-6, 9, dtype=torch.float64, device=b.device))
        levels = torch.cat([m * 2.0**-6, ((1 + m) * e[:, None]).reshape(-1)])[:-1]  # 0 to 448: the last pattern is NaN
        mid = (levels[1:] + levels[:-1]) / 2
        a = (unit.abs() * 448.0).contiguous()
        low, high = torch.bucketize(a, mid), torch.bucketize(a, mid, right=True)  # they differ at a tie alone
        v = torch.where(unit < 0, -1.0, 1.0) * levels[torch.where(low % 2 == 0, low, high)] * top / 448.0
    return v.reshape(y.shape[0], -1)[:, :y.shape[1]]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "norm":
        h = _exact_stream(s, c["p"]).to(torch.bfloat16).double()  # rounded by definition: what the residual stream holds
        mean = h.mean(1)
        rstd = ((h - mean[:, None]).square().mean(1) + EPS) ** -0.5
        y = (h - mean[:, None]) * rstd[:, None] * s["weight"].double() + s["bias"].double()
        if c["out"] != "bf16":
            y = _exact_codes(y.to(torch.bfloat16).double(), c["out"], c["group"])  # so is what is quantised
        return {"h": h, "mean": mean, "rstd": rstd, "y": y}
    if c["op"] == "norm_bwd":
        r = s["rstd"].double()[:, None]
        n = (s["h"].double() - s["mean"].double()[:, None]) * r
        dy = s["dy"].double()
        g = dy * s["weight"].double()
        dx = r * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
        if s["d_h"] is not None:
            dx = dx + s["d_h"].double()
        out = {"dx": dx, "dw": (dy * n).sum(0), "db": dy.sum(0)}
        if c["p"] > 0:
            out["dx_drop"] = _exact_dropped(dx, s["rng"], c["p"])
        return out
    if c["op"] == "dropout":
        return {"out": _exact_stream(s, c["p"])}
    x, w, H = s["x"].double(), s["w"].double(), c["H"]
    if c["op"] == "swiglu":
        gate, up = x @ w[:H].t(), x @ w[H:].t()
        out = {"y": gate * torch.sigmoid(gate) * up}
        if c["gu"]:
            out["gu"] = torch.cat([gate, up], 1)
        return out
    gate, up, dy = s["gu"][:, :H].double(), s["gu"][:, H:].double(), s["dy"].double()
    sig = torch.sigmoid(gate)
    d = torch.cat([dy * up * (sig + gate * sig * (1 - sig)), dy * gate * sig], 1).to(torch.bfloat16).double()  # rounded by definition
    return {"d_gu": d, "dx": d @ w, "dw": d.t() @ x}
