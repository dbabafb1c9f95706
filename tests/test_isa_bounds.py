"""Bounded stores in the gfx950 instructions of the norm and microscaled
operators (CPU only: hipcc compiles the sources with the library's flags).

A store through a buffer resource drops what lies at or past the record count.
The offset that is checked against it is the vector register's; what the scalar
register adds is documented as left out.  So a store that relies on the check
has its whole offset in the vector register.
"""

import re

import pytest

from test_isa_operators import SRC, _build, kernels, pytestmark  # noqa: F401

STORE = re.compile(r"(buffer_store_\w+)\s+\S+,\s*(\S+),\s*s\[\d+:\d+\],\s*(\S+)(.*)")


def scalar_offsets(lines):
    """The scalar offsets of the buffer stores of a kernel."""
    found = []
    for line in lines:
        if line.startswith("buffer_store"):
            m = STORE.match(line)
            assert m, line
            found.append(m.group(3))
    return found


@pytest.mark.parametrize("src", SRC)
def test_bounded_stores_have_no_scalar_offset(src):
    seen = 0
    for name, lines in kernels(_build.device_asm(src)).items():
        offsets = scalar_offsets(lines)
        assert set(offsets) <= {"0"}, (name, sorted(set(offsets)))
        seen += len(offsets)
    assert (seen > 0) == src.endswith("mxfp4.hip")


def test_the_check_sees_a_scalar_offset():
    assert scalar_offsets(["buffer_store_dword v1, v2, s[4:7], s9 offen"]) == ["s9"]
    assert scalar_offsets(["buffer_store_dword v1, v2, s[4:7], 0 offen"]) == ["0"]
