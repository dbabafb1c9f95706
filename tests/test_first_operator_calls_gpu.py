"""First calls of a process (GPU), each in a child process of its own.

* After prepare() no call of the library loads code: the number of code objects
  that the runtime's list for debuggers (`_amdgpu_r_debug`, a list in the form of
  the C library's r_debug) names does not change.
* The first call of a process can be captured into a HIP graph, for the norm,
  the quantiser, the product and the dequantisers as for the pass; the graph is
  replayed on two inputs, with eager work in between, and gives what eager calls
  of this process give.
"""

import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import swiglu_backward_int8_amd as sq

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
DEV = "cuda:0"
T, D, H, N = 128, 1024, 256, 512
SEEDS = (61, 62)


class _Link(ctypes.Structure):
    pass


_Link._fields_ = [("addr", ctypes.c_void_p), ("name", ctypes.c_char_p), ("ld", ctypes.c_void_p),
                  ("next", ctypes.POINTER(_Link)), ("prev", ctypes.POINTER(_Link))]


class _Debug(ctypes.Structure):
    _fields_ = [("version", ctypes.c_int), ("map", ctypes.POINTER(_Link))]


def code_objects():
    """How many code objects the process has loaded onto GPUs."""
    with open("/proc/self/maps") as f:
        paths = {line.split()[-1] for line in f if "libhsa-runtime64" in line}
    n = 0
    for path in paths:
        link = _Debug.in_dll(ctypes.CDLL(path), "_amdgpu_r_debug").map
        while link:
            n, link = n + 1, link.contents.next
    return n


def buffers():
    new = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device=DEV)
    bf16, f32, i8, u8 = torch.bfloat16, torch.float32, torch.int8, torch.uint8
    b = {"x": new(T, D, dtype=bf16), "r": new(T, D, dtype=bf16), "w": new(D, dtype=bf16), "dy": new(T, D, dtype=bf16)}
    b["W"] = new(N, D, dtype=bf16)
    out = {"q": new(T, D, dtype=i8), "s": new(T, D // 128, dtype=f32), "h": new(T, D, dtype=bf16), "rstd": new(T, dtype=f32),
           "y": new(T, D, dtype=bf16), "dx": new(T, D, dtype=bf16), "dw": new(D, dtype=f32), "v": new(T, D, dtype=bf16),
           "m": new(T, D, dtype=bf16), "C": new(T, N, dtype=f32), "one": new(1, N, dtype=bf16)}
    for name, (a, c) in (("a", sq.mxfp4_shapes(T, D)), ("at", sq.mxfp4_shapes(D, T)), ("b", sq.mxfp4_shapes(N, D))):
        out[name + "q"], out[name + "s"] = new(*a, dtype=u8), new(*c, dtype=u8)
    b["ws"] = sq.rms_norm_bwd_workspace(T, D, DEV)
    return b, out


def calls(b, o):
    sq.rms_norm_quant(b["x"], b["w"], o["q"], o["s"], residual=b["r"], h=o["h"], rstd=o["rstd"], y_bf16=o["y"])
    sq.group_dequant(o["q"], o["s"], o["v"])
    sq.mxfp4_quant(o["y"], o["aq"], o["as"], q_t=o["atq"], s_t=o["ats"])
    sq.mxfp4_quant(b["W"], o["bq"], o["bs"])
    sq.mxfp4_dequant(o["aq"], o["as"], o["m"])
    sq.mxfp4_gemm(o["aq"], o["as"], o["bq"], o["bs"], o["C"])
    sq.mxfp4_gemm(o["aq"][:1], o["as"][:1], o["bq"], o["bs"], o["one"])
    sq.rms_norm_bwd(b["dy"], o["h"], b["w"], o["rstd"], o["dx"], dw=o["dw"], workspace=b["ws"])


def fill(b, seed):
    g = torch.Generator().manual_seed(seed)
    for name in ("x", "r", "w", "dy", "W"):
        b[name].copy_(torch.randn(b[name].shape, generator=g))


def arrays(o):
    torch.cuda.synchronize()
    return {k: (t.view(torch.int16) if t.dtype is torch.bfloat16 else t).cpu().numpy() for k, t in o.items()}


def child_captures(path):
    b, o = buffers()
    torch.cuda.synchronize()
    print("capturing the first calls", flush=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(b, o)
    saved = {}
    for seed in SEEDS:
        fill(b, seed)
        for t in o.values():
            t.fill_(-7 if t.is_floating_point() or t.dtype is torch.int8 else 0xAA)
        graph.replay()
        saved.update(("%s_%d" % (k, seed), v) for k, v in arrays(o).items())
        print("replayed seed", seed, flush=True)
        calls(b, o)
    np.savez(path, **saved)


def child_counts():
    # what the runtime loads for itself, with the first launches and copies, first
    torch.zeros(8, device=DEV).cpu()
    b, o = buffers()
    x, dy = (torch.empty((T, n), dtype=torch.bfloat16, device=DEV) for n in (2 * H, H))
    outs, fp8 = sq.empty_outputs(T, H, DEV), sq.empty_outputs(T, H, DEV, fp8=True)
    a = torch.empty((T, H), dtype=torch.int8, device=DEV), torch.empty((T, H // 128), device=DEV)
    W, sW = torch.empty((N, D), dtype=torch.int8, device=DEV), torch.empty((N // 128, D // 128), device=DEV)
    torch.cuda.synchronize()
    before = code_objects()
    sq.prepare()
    prepared = code_objects()
    assert prepared > before, "prepare() loaded nothing: the list is not what this test takes it for"
    for what, call in (
            ("the pass", lambda: sq.silu_dot_fwd_bwd_quant_fuse(x, dy, *outs)),
            ("the E4M3 pass", lambda: sq.silu_dot_fwd_bwd_quant_fuse_fp8(x, dy, *fp8)),
            ("the forward quantiser", lambda: sq.silu_fwd_quant(x, *a)),
            ("the norm and the microscaled operators", lambda: calls(b, o)),
            ("the int8 product", lambda: sq.i8_gemm_group_scaled(o["q"], o["s"], W, sW, o["C"], b_rows_per_scale=128))):
        call()
        torch.cuda.synchronize()
        print("%s: %d code objects, %d when prepared, %d before" % (what, code_objects(), prepared, before), flush=True)
        assert code_objects() == prepared, what


def run_child(call):
    code = "import sys; sys.path[:0] = [%r, %r]; import test_first_operator_calls_gpu as t; t.%s" % (
        os.path.dirname(HERE), HERE, call)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]


def test_prepare_loads_the_code_of_every_operator():
    run_child("child_counts()")


def test_first_calls_captured_in_a_graph(tmp_path):
    path = str(tmp_path / "outs.npz")
    run_child("child_captures(%r)" % path)
    got = np.load(path)
    b, o = buffers()
    for seed in SEEDS:
        fill(b, seed)
        calls(b, o)
        for name, want in arrays(o).items():
            assert np.array_equal(got["%s_%d" % (name, seed)], want), (name, seed)
