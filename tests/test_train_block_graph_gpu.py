"""A captured training step of the example block, replayed with the step's number
changed on the device (GPU).  What the library makes of the step's inputs is compared
bit for bit with an eager step (torch's own products may add in another order inside a
capture), and what it makes of torch's products with eager calls on the same numbers."""

import pytest
import torch

import swiglu_backward_int8_amd as sq
from test_train_block_gpu import block, inputs, rng  # noqa: F401

pytestmark = pytest.mark.gpu

P = 0.2


def copied(t):
    """A copy made by a kernel, which a capture keeps as such."""
    return torch.bitwise_or(t.view(torch.int16), 0).view(t.dtype)


class Kept:
    """The library, keeping what its calls of a step read from torch's products and write."""

    def __init__(self):
        self.calls = {}

    def __getattr__(self, name):
        return getattr(sq, name)

    def layer_norm_quant(self, *args, **named):
        sq.layer_norm_quant(*args, **named)
        self.calls.update((k, named[k]) for k in ("h", "mean", "rstd"))
        self.calls["y"] = named["y_bf16"]

    def swiglu_gemm(self, y, w, a, gu):
        sq.swiglu_gemm(y, w, a, gu=gu)
        self.calls.update(a=a, gu=copied(gu))

    def dropout_add(self, x, out, p, rng, offset):
        if x is out:  # backward
            self.calls["d_ad"] = copied(x)
        sq.dropout_add(x, out, p, rng, offset=offset)
        self.calls["d_a" if x is out else "ad"] = out
        self.offset = offset

    def swiglu_gemm_bwd(self, dy, gu, x, w, d_gu, dx, dw, workspace):
        sq.swiglu_gemm_bwd(dy, gu, x, w, d_gu, dx=dx, dw=dw, workspace=workspace)
        self.calls.update(d_gu=d_gu, d_y=dx, d_w1=dw)

    def layer_norm_bwd(self, *args, **named):
        sq.layer_norm_bwd(*args, **named)
        self.calls.update(d_residual=args[5], dw=named["dw"], db=named["db"], d_x=named["dx_drop"])
        self.norm_offset = named["offset"]


FORWARD = ("h", "mean", "rstd", "y", "a", "gu", "ad")
BACKWARD = ("d_a", "d_gu", "d_y", "d_w1", "d_residual", "d_x", "dw", "db")


def backward(kept, args, state, D):
    """The library's backward calls, made eagerly on what torch's product gave the captured step."""
    x, residual, w, b, Wgu, Wd, d_out, d_h = args
    c = kept.calls
    out = {k: torch.empty_like(c[k]) for k in BACKWARD}
    T, H = c["a"].shape
    sq.dropout_add(c["d_ad"], out["d_a"], P, state, offset=kept.offset)
    sq.swiglu_gemm_bwd(out["d_a"], c["gu"], c["y"], Wgu, out["d_gu"], dx=out["d_y"], dw=out["d_w1"],
                       workspace=sq.swiglu_gemm_bwd_workspace(T, H, D, x.device))
    sq.layer_norm_bwd(out["d_y"], c["h"], w, c["mean"], c["rstd"], out["d_residual"], dw=out["dw"], db=out["db"], d_h=d_h,
                      dx_drop=out["d_x"], workspace=sq.layer_norm_bwd_workspace(T, D, x.device), p=P, rng=state, offset=kept.norm_offset)
    return out


@pytest.mark.parametrize("T,D,H", [(96, 256, 384), (33, 520, 264)])
def test_replays_are_eager_steps_bit_for_bit(block, monkeypatch, T, D, H):  # noqa: F811
    args, state = inputs(T, D, H, 3), rng(11, 0)
    steps = [0, 1, 2, 2**32 - 1]
    eager = []
    for step in steps:
        monkeypatch.setattr(block, "sq", Kept())
        state.copy_(torch.tensor([11, step]))
        block.train_bf16(*args, P, state)
        torch.cuda.synchronize()
        eager.append({k: t.clone() for k, t in block.sq.calls.items()})
    assert not torch.equal(eager[0]["ad"], eager[1]["ad"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # torch's products set themselves up outside a capture
        block.train_bf16(*args, P, state)
    torch.cuda.synchronize()
    kept = Kept()
    monkeypatch.setattr(block, "sq", kept)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.train_bf16(*args, P, state)
    for turn in (0, 1, 3, 2, 1, 0):
        state.copy_(torch.tensor([11, steps[turn]]))
        graph.replay()
        torch.cuda.synchronize()
        for k in FORWARD:
            assert torch.equal(kept.calls[k], eager[turn][k]), (turn, k)
        for k, want in backward(kept, args, state, D).items():
            assert torch.equal(kept.calls[k], want), (turn, k)
