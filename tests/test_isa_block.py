"""Checks of the gfx950 instructions generated for the layer norm, the dropout and the
gated projection (CPU only: hipcc compiles the sources with the library's flags).

* No packed fp32 arithmetic.
* The projection's kernels use no scratch memory and spill no vector registers: their
  waits for loads into LDS count memory operations.
* Nothing in front of a load into LDS breaks the wait states of its scalars, on any
  path (the check itself is tested with the microscaled product's).
* The matrix and the transposing LDS instructions are there.
"""

import re

import pytest

import isa
from test_isa_waits import hazards, pytestmark  # noqa: F401


@pytest.mark.parametrize("source", ["layernorm", "swiglugemm"])
def test_no_packed_fp32(source):
    assert isa.kernels(source)
    assert not re.search(r"\bv_pk_(fma|mul|add)_f32\b", isa.text(source))


def test_no_scratch_and_no_spilled_vector_registers():
    found = isa.metadata("swiglugemm")
    assert set(found) == set(isa.kernels("swiglugemm"))
    for name, (scratch, vectors, _) in found.items():
        assert scratch == 0 and vectors == 0, name
    for name, (scratch, vectors, _) in isa.metadata("layernorm").items():
        # rows of more than 8192 columns in 128 registers a lane: a few of the backward pass's
        if "layer_norm_bwd_kernelILb0ELi2ELi1024E" in name:
            assert scratch <= 128, (name, scratch)
        else:
            assert scratch == 0 and vectors == 0, name


def test_loads_into_lds_wait_for_their_scalars_on_every_path():
    total = 0
    for name, kernel in isa.kernels("swiglugemm").items():
        bad, loads = hazards(kernel)
        assert not bad, (name, bad[:3])
        total += loads
    assert total > 1000


def test_instructions():
    tiles = {n: k for n, k in isa.kernels("swiglugemm").items() if "swiglu_tile_kernel" in n}
    assert len(tiles) == 2 * 4 + 2 * 4 + 2 * 3  # gated (with and without gu), dx and dw (bf16 and fp32), by their tiles
    for name, kernel in tiles.items():
        ops = [op for op, _ in kernel.code]
        assert ops.count("v_mfma_f32_32x32x16_bf16") >= 4 * 2, name
        by_k = "ProductE0" not in name
        assert ("ds_read_b64_tr_b16" in ops) == by_k, name
        assert any(isa.into_lds(*c) and c[0] == "buffer_load_dwordx4" for c in kernel.code), name
    stream = [k for n, k in isa.kernels("swiglugemm").items() if "swiglu_stream_kernel" in n]
    assert len(stream) == 2
    for kernel in stream:
        ops = [op for op, _ in kernel.code]
        assert "v_mfma_f32_16x16x32_bf16" in ops and "global_load_dwordx4" in ops
