"""No barrier is passed with LDS operations still on their way, in the gfx950
instructions that the compiler made (CPU only).

What a wave writes to LDS is there for the others, or out of their way, behind a
barrier if the wave has waited for it in front of it.  The compiler's own waits do not
cover every path: where a wave skips the reads behind its writes (nothing of a tile to
store), none was left in front of the next tile's barrier.  LDS operations are carried
out in their order, so a wait for at most N ends all but the N newest; scalar loads
counted with them only make it wait longer."""

import re

import pytest

import isa
from test_isa_waits import pytestmark  # noqa: F401

SOURCES = ["siluquant", "i8gemm", "rmsnorm", "mxfp4", "mxfp4gemm", "layernorm", "swiglugemm"]


def pending(kernel, which=r"ds_"):
    """The barriers that some path reaches with an operation of `which` not waited for."""
    none = 99
    after = [[] for _ in kernel.code]
    for i, before in enumerate(kernel.before):
        for b in before:
            after[b].append(i)
    # per instruction: LDS operations issued behind the newest one that may still be on its way; none: there is none
    state, todo, found = {0: none}, [0], set()
    while todo:
        i = todo.pop()
        newer, (op, args) = state[i], kernel.code[i]
        if op == "s_barrier" and newer != none:
            found.add(i)
        if op == "s_waitcnt":
            count = re.search(r"lgkmcnt\((\d+)\)", " ".join(args))
            if count and int(count.group(1)) <= newer:
                newer = none
        elif re.match(which, op):
            newer = 0
        elif op.startswith("ds_") and newer != none:
            newer = min(newer + 1, 15)
        for j in after[i]:
            if newer < state.get(j, none + 1):
                state[j] = newer
                todo.append(j)
    return sorted(found)


@pytest.mark.parametrize("source", SOURCES)
def test_nothing_is_on_its_way_at_a_barrier(source):
    barriers = 0
    for name, kernel in isa.kernels(source).items():
        assert not pending(kernel), name
        barriers += sum(op == "s_barrier" for op, _ in kernel.code)
    assert barriers > 0


def test_the_check_follows_paths():
    write, read, wait = "ds_write_b128 v1, v[2:5]", "ds_read_b128 v[2:5], v1", "s_waitcnt lgkmcnt(%d)"
    found = lambda *lines, which=r"ds_": bool(pending(isa.Kernel(lines + ("s_barrier", "s_endpgm")), which))
    assert found(write) and not found(write, wait % 0) and found(write, wait % 1)
    assert found(write, "s_waitcnt vmcnt(0)") and not found(write, "s_waitcnt vmcnt(0) lgkmcnt(0)")
    assert found(write, read, wait % 1) and not found(write, read, wait % 1, which=r"ds_write")
    assert found(write, "s_cbranch_execz .L1", read, wait % 0, ".L1:")
    assert not found(write, "s_cbranch_execz .L1", read, ".L1:", wait % 0)
    assert found(".L1:", "s_barrier", write, "s_cbranch_scc1 .L1", wait % 0)
