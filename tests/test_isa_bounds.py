"""Bounded stores in the gfx950 instructions of the norm and microscaled
operators (CPU only).

A store through a buffer resource drops what lies at or past the record count.
The offset that is checked against it is the vector register's; what the scalar
register adds is documented as left out.  So a store that relies on the check
has its whole offset in the vector register.
"""

import pytest

import isa
from test_isa_waits import pytestmark  # noqa: F401


def scalar_offsets(kernel):
    """The scalar offsets of the buffer stores of a kernel."""
    return [args[3].split()[0] for op, args in kernel.code if op.startswith("buffer_store")]


@pytest.mark.parametrize("source", isa.OPERATORS)
def test_bounded_stores_have_no_scalar_offset(source):
    seen = 0
    for name, kernel in isa.kernels(source).items():
        offsets = scalar_offsets(kernel)
        assert set(offsets) <= {"0"}, (name, sorted(set(offsets)))
        seen += len(offsets)
    assert (seen > 0) == (source == "mxfp4")


def test_the_check_sees_a_scalar_offset():
    assert scalar_offsets(isa.Kernel(["buffer_store_dword v1, v2, s[4:7], s9 offen"])) == ["s9"]
    assert scalar_offsets(isa.Kernel(["buffer_store_dword v1, v2, s[4:7], 0 offen"])) == ["0"]
