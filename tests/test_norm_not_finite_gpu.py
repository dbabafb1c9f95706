"""Values that are not finite in the norm's output (GPU): what the group's scale
shows, and that nothing else changes."""

import pytest
import torch

from test_rms_norm_gpu import inputs, run_forward

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("D", [384, 2050])
def test_infinite_y_gives_an_infinite_scale(D, e4m3):
    x, r, w = inputs(4, D, False, True, seed=2)
    want = run_forward(x, r, w, 128, e4m3)
    w = w.clone()
    w[200] = INF
    q, s, y, h, rstd = run_forward(x, r, w, 128, e4m3)
    assert torch.equal(h, want[3]) and torch.equal(rstd, want[4])
    hit = h[:, 200] != 0  # inf * 0 is NaN
    assert hit.any() and bool(torch.isinf(y[hit, 200]).all())
    assert bool((s[hit, 1] == INF).all()) and bool(torch.isnan(s[~hit, 1]).all())
    groups = [g for g in range(s.shape[1]) if g != 1]
    assert torch.equal(s[:, groups], want[1][:, groups])
    cols = [c for c in range(D) if c // 128 != 1]
    bits = lambda t: t.view(torch.uint8)[:, cols]
    assert torch.equal(bits(q), bits(want[0]))


@pytest.mark.parametrize("D", [384, 2050, 20000])
def test_rows_of_h_that_are_not_finite(D):
    x, r, w = inputs(5, D, False, True, seed=3)
    x, r = x.clone(), r.clone()
    x[1], x[3], r[1], r[3] = 1.0, 1.0, 0.0, 0.0  # rows without zeros
    want = run_forward(x, r, w, 128, False)
    x[1, 130], x[3, 130] = INF, NAN
    q, s, y, h, rstd = run_forward(x, r, w, 128, False)
    assert rstd[1] == 0 and torch.isnan(rstd[3])
    assert torch.isnan(y[1, 130]) and bool((y[1, :130] == 0).all()) and bool((y[1, 131:] == 0).all())
    assert torch.isnan(s[1, 1]) and s[1, 0] == 1 and bool((s[1, 2:] == 1).all()) and bool((q[1, :128] == 0).all())
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isnan(s[3]).all())
    for a, b in zip((q, s, y, h, rstd), want):
        assert torch.equal(a[[0, 2, 4]], b[[0, 2, 4]])
