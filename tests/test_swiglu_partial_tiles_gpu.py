"""Tiles of a few rows, in front of whole ones that the same workgroup takes next (GPU):
most of its waves have nothing to store there.  Small whole numbers, equal to the last
bit, several times each, since what one wave leaves to another depends on their timing."""

import pytest
import torch

import plans
import test_swiglu_gemm_gpu as gemm

pytestmark = pytest.mark.gpu

# the product and the tiles that a size is for: its last row of tiles has 5 to 16 rows
SHAPES = {
    (773, 7648, 168): ("gated", "k128Two"), (773, 7680, 192): ("gated", "k128Two"), (773, 7648, 104): ("gated", "k128Two"),
    (264, 11952, 16): ("gated", "k128Two"), (3713, 2280, 592): ("gated", "k128"), (21762, 528, 208): ("gated", "k256"),
    (136, 9976, 1240): ("gated", "k64"),
    (2184, 328, 7288): ("dx", "k128"), (27016, 16, 272): ("dx", "k128Two"), (15109, 128, 1552): ("dx", "k256"), (387, 1200, 9152): ("dx", "k64"),
    (582, 1736, 4616): ("dw", "k128"), (5, 11592, 272): ("dw", "k128Two"), (249, 5768, 2144): ("dw", "k256"),
}
TIMES = 6


def planned(shape):
    """The tiles of the product that a size is for, and whether whole tiles follow partial ones in a workgroup."""
    product, tiles = SHAPES[shape]
    T, H, D = shape
    M, columns = {"gated": (T, 2 * H), "dx": (T, D), "dw": (2 * H, D)}[product]
    turns = plans.sequences(tiles, M, columns)
    return (product, tiles, 1, True) in plans.kernels([shape])[0], any(p == (False, True) for t in turns for p in zip(t, t[1:]))


@pytest.mark.parametrize("T,H,D", [s for s in SHAPES if SHAPES[s][0] == "gated"])
def test_forward(T, H, D):
    assert planned((T, H, D)) == (True, True)
    x, w = gemm.whole(T, H, D, T + H)
    want = (x.double() @ w.double().t()).to(torch.bfloat16)
    first, _ = gemm.run_forward(x, w)
    for i in range(TIMES):
        y, gu = gemm.run_forward(x, w)
        assert torch.equal(gu, want) and torch.equal(y, first), i
        assert torch.equal(gemm.run_forward(x, w, gu=False)[0], first), i


@pytest.mark.parametrize("T,H,D", [s for s in SHAPES if SHAPES[s][0] != "gated"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_backward(T, H, D, dtype):
    assert planned((T, H, D)) == (True, True)
    dy, gu, x, w = gemm.whole_backward(T, H, D, T + H)
    gate, up = gu.double().chunk(2, 1)
    d = torch.cat([dy.double() * up * torch.where(gate == 0, 0.5, 1.0), dy.double() * torch.where(gate == 0, 0.0, gate)], 1)
    want = (d @ w.double()).to(dtype), (d.t() @ x.double()).to(dtype)
    for i in range(TIMES):
        d_gu, dx, dw = gemm.run_backward(dy, gu, x, w, dtype, dtype)
        assert torch.equal(d_gu.double(), d), i
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1]), i
