"""Which kernels of the norm are compiled (CPU only): none that no call reaches."""

import isa
from test_isa_waits import pytestmark  # noqa: F401


def pieces_and_kind(name):
    """(pieces per lane, kind) of a norm kernel with those template arguments, or None."""
    for kernel in ("rms_norm_quant_kernelILb", "rms_norm_bwd_kernelILb"):
        if kernel in name:
            rest = name.split(kernel)[1]
            return int(rest.split("ELi")[1][0]), int(rest.split("KindE")[1][0])
    return None


def test_short_rows_have_one_piece_per_lane():
    # rows of fewer than 8 columns (kind 3) go to a wave with one piece per lane;
    # two pieces start at 513 columns
    found = [pieces_and_kind(n) for n in isa.kernels("rmsnorm")]
    found = [f for f in found if f]
    assert (1, 3) in found and (2, 2) in found
    assert (2, 3) not in found
