"""The backward norm looks at its workspace only where it needs one (GPU):
without dw, and up to 16384 columns, whatever is given for it is left alone."""

import pytest
import torch

import swiglu_backward_int8_amd as sq
from test_rms_norm_gpu import DEV, bwd_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D", [(8, 256), (3, 2050)])
def test_workspace_is_not_looked_at_without_dw(T, D):
    dy, h, w, rstd, d_h = (t.to(DEV) for t in bwd_inputs(T, D, False, True, seed=1))
    want, dx = torch.empty_like(h), torch.empty_like(h)
    sq.rms_norm_bwd(dy, h, w, rstd, want, d_h=d_h)
    room = torch.full((sq.rms_norm_bwd_workspace(T, D, DEV).numel() + 1,), 0x5A, dtype=torch.uint8, device=DEV)
    before = h.clone()
    # too small, off 16 bytes, and an input's own memory
    for ws in (room[:16], room[1:], h.view(torch.uint8)):
        dx.fill_(float("nan"))
        sq.rms_norm_bwd(dy, h, w, rstd, dx, d_h=d_h, workspace=ws)
        assert torch.equal(dx, want)
    assert torch.equal(h, before) and bool((room == 0x5A).all())


def test_workspace_is_looked_at_where_it_is_needed():
    dy, h, w, rstd, d_h = (t.to(DEV) for t in bwd_inputs(8, 256, False, True, seed=1))
    dx, dw = torch.empty_like(h), torch.empty(256, device=DEV)
    room = torch.empty(sq.rms_norm_bwd_workspace(8, 256, DEV).numel() + 1, dtype=torch.uint8, device=DEV)
    for ws in (None, room[:16], room[1:], h.view(torch.uint8)):
        with pytest.raises(ValueError):
            sq.rms_norm_bwd(dy, h, w, rstd, dx, dw=dw, d_h=d_h, workspace=ws)
