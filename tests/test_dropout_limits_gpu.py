"""dropout_add past 2^29 pieces of eight columns, where it launches again, and past
the 2^32 threads that a launch may have (GPU).  Rows at the ends, and on both sides of
the second launch's first piece, are compared with the oracle's."""

import pytest
import torch

import ln64
import swiglu_backward_int8_amd as sq
from test_block_limits_gpu import DEV, RNG, kept_rows, rng

pytestmark = pytest.mark.gpu

bf16, f32 = torch.bfloat16, torch.float32
ROWS = 40


@pytest.fixture(autouse=True)
def _memory():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def places(T, D):
    again = 2**29 // -(-D // 8)  # the row of the first piece past 2^20 workgroups' 512
    return [0, again - ROWS // 2, T // 3, T - ROWS]


@pytest.mark.parametrize("T,D", [(2**29 + 77, 1), (2**29 + 5000, 8), (2**27 + 77, 25), (2**31, 25)])
def test_in_place(T, D):
    print("dropout in place", T, D, flush=True)
    x = torch.ones((T, D), dtype=bf16, device=DEV)
    sq.dropout_add(x, x, 0.25, rng())
    factor = torch.tensor(ln64.scale(0.25)).to(bf16)
    for first in places(T, D):
        want = torch.where(kept_rows(first, ROWS, D, 0.25), factor, torch.zeros_like(factor))
        assert torch.equal(x[first:first + ROWS].cpu(), want), first


@pytest.mark.parametrize("T,D", [(2**29 + 77, 3), (2**27 + 77, 26), (2**26 + 77, 64)])
def test_fp32_with_a_residual(T, D):
    print("dropout of fp32 with a residual", T, D, flush=True)
    g = torch.Generator(device=DEV).manual_seed(D)
    x, r = torch.full((T, D), 0.5, device=DEV), torch.full((T, D), -2.0, dtype=bf16, device=DEV)
    for first in places(T, D):
        x[first:first + ROWS] = torch.randn((ROWS, D), generator=g, device=DEV)
        r[first:first + ROWS] = torch.randn((ROWS, D), generator=g, device=DEV).to(bf16)
    out = torch.full((T, D), float("nan"), dtype=bf16, device=DEV)
    sq.dropout_add(x, out, 0.25, rng(), residual=r)
    assert not torch.isnan(out.view(-1)[::1021].float()).any()
    for first in places(T, D):
        rows = slice(first, first + ROWS)
        v = torch.where(kept_rows(first, ROWS, D, 0.25), x[rows].cpu() * ln64.scale(0.25), torch.zeros(()))
        assert torch.equal(out[rows].cpu(), (r[rows].cpu().float() + v).to(bf16)), first


def test_captured():
    # a call of several launches is captured whole, and draws anew when the numbers change
    T, D = 2**29 + 77, 1
    x, out, numbers = torch.ones((T, D), dtype=bf16, device=DEV), torch.empty((T, D), dtype=bf16, device=DEV), rng()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sq.dropout_add(x, out, 0.25, numbers)
    eager = torch.empty_like(out)
    for step in (5, 6, 5):
        numbers.copy_(torch.tensor([RNG[0], step]))
        out.fill_(7)
        graph.replay()
        sq.dropout_add(x, eager, 0.25, numbers)
        torch.cuda.synchronize()
        assert torch.equal(out, eager), step
        assert torch.equal((out[:ROWS] != 0).cpu(), ln64.kept((RNG[0], step), ROWS, D, 0.25)), step
