"""Checks of the gfx950 instructions generated for the layer norm, the dropout and the
gated projection (CPU only: hipcc compiles the sources with the library's flags).

* No packed fp32 arithmetic.
* The projection's kernels use no scratch memory and spill no vector registers: their
  waits for loads into LDS count memory operations.
* Nothing in front of a load into LDS breaks the wait states of its scalars, on any
  path (the check itself is tested with the microscaled product's).
* A tile's start waits until no more than N memory operations are left, in the order of
  their issue, where the tile before it was whole: at least N stores come after the last
  of its loads into LDS.
* The matrix and the transposing LDS instructions are there.
"""

import re

import pytest

import isa
from test_isa_waits import counted_waits, hazards, pytestmark  # noqa: F401


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


def stores_behind_the_loads(kernel):
    """For each run of instructions without a branch that loads into LDS and stores after
    that (a whole tile's end): the stores after its last load."""
    out = []
    for block in kernel.blocks():
        loads = [i for i, c in enumerate(block) if isa.into_lds(*c)]
        behind = sum(op == "global_store_dwordx4" for op, _ in block[loads[-1]:]) if loads else 0
        out += [behind] if behind else []
    return out


def test_stores_that_the_tiles_do_not_wait_for():
    for name, kernel in isa.kernels("swiglugemm").items():
        if "swiglu_tile_kernel" in name:
            # the loop's count, where loads are left on their way, stands with one of LDS operations
            waits, stores = counted_waits(kernel), stores_behind_the_loads(kernel)
            assert len(waits) == 1 and len(stores) == 1, (name, waits, stores)
            assert stores[0] >= waits[0] > 0, (name, waits, stores)


def test_the_count_sees_a_store_too_few():
    load, store, branch = "buffer_load_dwordx4 v1, s[4:7], 0 offen lds", "global_store_dwordx4 v[2:3], v[4:7], off", "s_cbranch_scc1 .L1"
    lines = [".L1:", load, branch, load, store, store, load, store, store, branch, store, "s_endpgm"]
    assert stores_behind_the_loads(isa.Kernel(lines)) == [2]
    assert stores_behind_the_loads(isa.Kernel(lines[:7] + lines[8:])) == [1]
    assert stores_behind_the_loads(isa.Kernel(lines[:9] + [load] + lines[9:])) == []


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
    assert len(stream) == 2 * 3  # with and without gu, by the rows of x
    for kernel in stream:
        ops = [op for op, _ in kernel.code]
        assert "v_mfma_f32_16x16x32_bf16" in ops and "global_load_dwordx4" in ops
