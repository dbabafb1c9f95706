"""What the product kernels' hand-written waits rest on, in the gfx950
instructions that the compiler made (CPU only).

* The tiles' counted wait.  A tile's first loads into LDS are issued before the
  stores of the tile before it, and its start waits until no more than N memory
  operations are left, in the order of their issue.  That covers the loads as
  long as at least N stores come after the last of them, on both ways (streamed
  and not) that a whole tile is stored.
* Wait states in front of the loads into LDS, along every path, the loops' back
  edges among them: five after a vector instruction's write of a scalar register
  that the load reads, one after any write of M0.
* No kernel uses scratch memory or spills vector registers (a spilled scalar goes
  to a vector register's lanes; a reload of it would be a memory operation that
  the waits do not count if it went to scratch).
"""

import os
import shutil

import pytest

import isa
from swiglu_backward_int8_amd import _build

pytestmark = pytest.mark.skipif(not os.path.exists(_build.hipcc()) and shutil.which("hipcc") is None,
                                reason="hipcc is not installed")


def counted_waits(kernel):
    """The counts above zero of the waits for memory operations alone."""
    return [int(args[0][6:-1]) for op, args in kernel.code
            if op == "s_waitcnt" and len(args) == 1 and args[0].startswith("vmcnt(") and " " not in args[0]
            and args[0] != "vmcnt(0)"]


def stores_after_the_loads(kernel):
    """For each run of instructions that loads into LDS and stores whole chunks without a
    branch (a whole tile's end): the stores after its last load."""
    out = []
    for block in kernel.blocks():
        loads = [i for i, (op, args) in enumerate(block) if isa.into_lds(op, args)]
        stores = [i for i, (op, _) in enumerate(block) if op == "global_store_dwordx4"]
        if loads and len(stores) >= 8:
            out.append(sum(i > loads[-1] for i in stores))
    return out


def tiles_with_counted_waits():
    # template arguments: blocks of rows of A and of B, waves, buffers, exponents in words, bf16 results
    return {n: k for n, k in isa.kernels("mxfp4gemm").items() if "mx_gemm_tile_kernel" in n and "ELb1ELb" in n}


def test_stores_that_the_tiles_do_not_wait_for():
    found = tiles_with_counted_waits()
    assert len(found) == 6
    for name, kernel in found.items():
        waits, stores = counted_waits(kernel), stores_after_the_loads(kernel)
        assert len(waits) == 1 and len(stores) == 2, (name, waits, stores)
        assert min(stores) >= waits[0], (name, waits, stores)


def test_the_count_sees_a_store_too_few():
    # the same instructions with the last store of either way left out, and with a load after it
    name, kernel = next(iter(tiles_with_counted_waits().items()))
    asm = isa.text("mxfp4gemm")
    start = asm.index("\n%s:" % name)
    lines = asm[start:asm.find(".Lfunc_end", start)].splitlines()
    want = counted_waits(kernel)[0]
    stores = [i for i, l in enumerate(lines) if l.strip().startswith("global_store_dwordx4")]
    last = [i for i in stores if i + 1 == len(lines) or not any(
        i < j <= i + 400 and not any(l.strip().startswith(("s_branch", "s_cbranch")) for l in lines[i:j]) for j in stores)]
    seen = 0
    for i in last:
        fewer = stores_after_the_loads(isa.Kernel(lines[:i] + lines[i + 1:]))
        later = stores_after_the_loads(isa.Kernel(
            lines[:i + 1] + ["buffer_load_dwordx4 v1, s[4:7], 0 offen lds"] + lines[i + 1:]))
        seen += min(fewer, default=want) < want and min(later) == 0
    assert seen >= 2


def hazards(kernel):
    """(write, load) pairs with too few wait states between them on some path, and the number of loads."""
    bad, loads = [], 0
    for i, (op, args) in enumerate(kernel.code):
        if not isa.into_lds(op, args):
            continue
        loads += 1
        reads = set().union(*(isa.scalars(a) for a in args))
        todo, done = [(p, 0) for p in kernel.before[i]], set()
        while todo:
            at, states = todo.pop()
            if states >= 5 or (at, states) in done:
                continue
            done.add((at, states))
            p, pargs = kernel.code[at]
            writes = isa.written(p, pargs)
            if (p.startswith("v_") and writes & reads) or ("m0" in writes and states < 1):
                bad.append(((p, pargs), (op, args)))
            states += int(pargs[0]) + 1 if p == "s_nop" else 1
            todo += [(b, states) for b in kernel.before[at]]
    return bad, loads


@pytest.mark.parametrize("source", ["mxfp4gemm", "i8gemm"])
def test_loads_into_lds_wait_for_their_scalars_on_every_path(source):
    total = 0
    for name, kernel in isa.kernels(source).items():
        bad, loads = hazards(kernel)
        assert not bad, (name, bad[:3])
        total += loads
    assert total > 100


def test_the_hazard_check_follows_paths():
    load = "buffer_load_dwordx4 v1, s[4:7], s9 offen lds"
    found = lambda *lines: bool(hazards(isa.Kernel(lines + ("s_endpgm",)))[0])
    assert found("v_readlane_b32 s6, v9, 1", "s_nop 0", load)
    assert not found("v_readlane_b32 s6, v9, 1", "s_nop 4", load)
    assert not found("v_readlane_b32 s3, v9, 1", load)
    assert found("v_cmp_eq_u32_e64 s[8:9], v1, v2", "s_nop 2", load)
    assert found("v_add_co_u32_e64 v1, s[8:9], v1, v2", load)
    assert found("s_mov_b32 m0, s2", load) and not found("s_mov_b32 m0, s2", "s_nop 0", load)
    assert found("s_add_i32 m0, s2, 16", load) and found("v_readfirstlane_b32 m0, v2", load)
    assert not found("s_mov_b32 s9, s2", load)
    # written at a loop's end, read at its start; and behind a branch that is taken
    assert found(".L1:", load, "s_nop 7", "v_readfirstlane_b32 s9, v3", "s_cbranch_scc1 .L1")
    assert not found(".L1:", load, "v_readfirstlane_b32 s9, v3", "s_nop 4", "s_cbranch_scc1 .L1")
    assert found("v_readfirstlane_b32 s9, v3", "s_branch .L2 ; a comment", "s_nop 7", ".L2:  ; another", load)


@pytest.mark.parametrize("source", isa.OPERATORS)
def test_no_scratch_and_no_spilled_vector_registers(source):
    found = isa.metadata(source)
    assert set(found) == set(isa.kernels(source))
    for name, (scratch, vectors, _) in found.items():
        assert scratch == 0 and vectors == 0, name
