"""First calls, captures, streams and threads of the layer norm, the dropout and the
gated projection (GPU)."""

import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import swiglu_backward_int8_amd as sq
import test_first_operator_calls_gpu as first

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
T, D, H = 100, 512, 264
SEEDS = (61, 62)
bf16, f32 = torch.bfloat16, torch.float32


def buffers():
    new = lambda *shape, dtype=bf16: torch.empty(shape, dtype=dtype, device=DEV)
    b = {"x": new(T, D), "r": new(T, D), "w": new(D), "b": new(D), "W": new(2 * H, D), "dy": new(T, H), "d_h": new(T, D)}
    b["rng"] = torch.tensor([5, 6], dtype=torch.int64, device=DEV)
    b["ws"] = sq.swiglu_gemm_bwd_workspace(T, H, D, DEV)
    b["wn"] = sq.layer_norm_bwd_workspace(T, D, DEV)
    out = {"h": new(T, D), "y": new(T, D), "mean": new(T, dtype=f32), "rstd": new(T, dtype=f32), "q": new(T, D, dtype=torch.int8),
           "s": new(T, D // 128, dtype=f32), "a": new(T, H), "gu": new(T, 2 * H), "one": new(1, H), "ad": new(T, H), "d_gu": new(T, 2 * H),
           "d_y": new(T, D, dtype=f32), "dW": new(2 * H, D), "dr": new(T, D), "dx": new(T, D), "dw": new(D, dtype=f32), "db": new(D, dtype=f32)}
    return b, out


def calls(b, o):
    sq.layer_norm_quant(b["x"], b["w"], b["b"], o["q"], o["s"], residual=b["r"], h=o["h"], mean=o["mean"], rstd=o["rstd"], y_bf16=o["y"],
                        p=0.1, rng=b["rng"])
    sq.swiglu_gemm(o["y"], b["W"], o["a"], gu=o["gu"])
    sq.swiglu_gemm(o["y"][:1], b["W"], o["one"])
    sq.dropout_add(o["a"], o["ad"], 0.2, b["rng"], offset=1)
    sq.swiglu_gemm_bwd(b["dy"], o["gu"], o["y"], b["W"], o["d_gu"], dx=o["d_y"], dw=o["dW"], workspace=b["ws"])
    sq.layer_norm_bwd(o["d_y"], o["h"], b["w"], o["mean"], o["rstd"], o["dr"], dw=o["dw"], db=o["db"], d_h=b["d_h"], dx_drop=o["dx"],
                      workspace=b["wn"], p=0.1, rng=b["rng"])


def fill(b, seed):
    g = torch.Generator().manual_seed(seed)
    for name in ("x", "r", "w", "b", "W", "dy", "d_h"):
        b[name].copy_(torch.randn(b[name].shape, generator=g))
    b["rng"].copy_(torch.tensor([seed, 3]))


def clear(o):
    for t in o.values():
        t.fill_(-7)


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
        clear(o)
        graph.replay()
        saved.update(("%s_%d" % (k, seed), v) for k, v in first.arrays(o).items())
        print("replayed seed", seed, flush=True)
        calls(b, o)
    np.savez(path, **saved)


def child_counts():
    torch.zeros(8, device=DEV).cpu()
    b, o = buffers()
    fill(b, 1)
    torch.cuda.synchronize()
    before = first.code_objects()
    sq.prepare()
    prepared = first.code_objects()
    assert prepared > before
    calls(b, o)
    torch.cuda.synchronize()
    print("%d code objects, %d when prepared, %d before" % (first.code_objects(), prepared, before), flush=True)
    assert first.code_objects() == prepared


def run_child(call):
    code = "import sys; sys.path[:0] = [%r, %r]; import test_block_calls_gpu as t; t.%s" % (
        first.os.path.dirname(first.HERE), first.HERE, call)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]


def test_prepare_loads_the_code():
    run_child("child_counts()")


def test_first_calls_captured_in_a_graph(tmp_path):
    path = str(tmp_path / "outs.npz")
    run_child("child_captures(%r)" % path)
    got = np.load(path)
    b, o = buffers()
    for seed in SEEDS:
        fill(b, seed)
        calls(b, o)
        for name, want in first.arrays(o).items():
            assert np.array_equal(got["%s_%d" % (name, seed)], want, equal_nan=True), (name, seed)


def test_two_graphs_share_workspaces():
    # on one stream, in turn: neither leaves anything in them that the other reads
    b, o = buffers()
    b2, o2 = buffers()
    b2["ws"], b2["wn"] = b["ws"], b["wn"]
    graphs, wants = [], []
    for seed, (bb, oo) in zip(SEEDS, ((b, o), (b2, o2))):
        fill(bb, seed)
        calls(bb, oo)
        wants.append({k: t.clone() for k, t in oo.items()})
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            calls(bb, oo)
        graphs.append(graph)
    for turn in (0, 1, 1, 0, 1, 0):
        clear((o, o2)[turn])
        b["ws"].fill_(0xff), b["wn"].fill_(0xff)
        graphs[turn].replay()
        torch.cuda.synchronize()
        for k, t in (o, o2)[turn].items():
            assert torch.equal(t, wants[turn][k]), (turn, k)


def test_two_streams_and_two_threads():
    # each with buffers of its own: the library keeps nothing between calls
    sets = [buffers() for _ in range(3)]
    wants = []
    for seed, (b, o) in enumerate(sets):
        fill(b, seed)
        calls(b, o)
        torch.cuda.synchronize()
        wants.append({k: t.clone() for k, t in o.items()})
        clear(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        for stream, (b, o) in zip(streams, sets):
            with torch.cuda.stream(stream):
                calls(b, o)
    torch.cuda.synchronize()
    for want, (b, o) in zip(wants, sets):
        assert all(torch.equal(t, want[k]) for k, t in o.items())
        clear(o)
    torch.cuda.synchronize()
    failed = []

    def work(stream, b, o):
        try:
            with torch.cuda.stream(stream):
                for _ in range(5):
                    calls(b, o)
        except Exception as e:  # a thread's exception would be lost
            failed.append(e)

    threads = [threading.Thread(target=work, args=(s, b, o)) for s, (b, o) in zip(streams, sets)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for want, (b, o) in zip(wants, sets):
        assert all(torch.equal(t, want[k]) for k, t in o.items())


def test_workspaces_are_looked_at_only_where_they_are_needed():
    b, o = buffers()
    fill(b, 1)
    calls(b, o)
    room = torch.full((1 << 20,), 0x5A, dtype=torch.uint8, device=DEV)
    dx, gu = torch.empty_like(o["dr"]), torch.empty_like(o["gu"])
    for ws in (None, room[:16], room[1:], o["h"].view(torch.uint8)):
        sq.layer_norm_bwd(o["d_y"], o["h"], b["w"], o["mean"], o["rstd"], dx, d_h=b["d_h"], workspace=ws)
        assert torch.equal(dx, o["dr"])
        sq.swiglu_gemm_bwd(b["dy"], o["gu"], o["y"], b["W"], gu, workspace=ws)
        assert torch.equal(gu, o["d_gu"])
    assert bool((room == 0x5A).all())
    big_h, big_d = 5504, 256  # sums long enough for slices
    t = lambda *s: torch.zeros(s, dtype=bf16, device=DEV)
    need = sq.swiglu_gemm_bwd_workspace(64, big_h, big_d, DEV)
    assert need.numel() > 0
    for ws in (None, need[:-16], room[1:need.numel() + 1]):
        with pytest.raises(ValueError):
            sq.swiglu_gemm_bwd(t(64, big_h), t(64, 2 * big_h), t(64, big_d), t(2 * big_h, big_d), t(64, 2 * big_h), dx=t(64, big_d),
                               workspace=ws)
