"""The ends of the sizes that dropout_add takes: refused past them, and not before
(CPU only: the calls that are not refused for their size are for a null pointer)."""

import pytest

import swiglu_backward_int8_amd as sq
from test_operators_abi import at, caller


@pytest.fixture(scope="module")
def dropout():
    names = "x x_dtype residual out T D p rng offset stream".split()
    return caller(sq.lib().dropout_add, names, (at(0), 1, None, at(0), 8, 256, 0.1, at(3), 0, None))


@pytest.mark.parametrize("T,D", [(2**31, 513), (2**31, 4088), (2**28 + 1, 4096), (2**18 + 1, 2**22), (2**31, 2**22)])
def test_more_than_2_to_the_40_elements_are_refused(dropout, T, D):
    assert dropout(T=T, D=D) == 2
    assert dropout(T=T, D=D, out=None) == 2


@pytest.mark.parametrize("T,D", [(2**31, 512), (2**31, 25), (2**31, 1), (2**28, 4096), (2**18, 2**22)])
def test_up_to_2_to_the_40_elements_are_taken(dropout, T, D):
    assert dropout(T=T, D=D, x=None) == 1 and dropout(T=T, D=D, out=None) == 1
