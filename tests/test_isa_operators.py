"""Checks of the gfx950 instructions generated for the norm and microscaled
operators (CPU only: hipcc compiles the sources with the library's flags).

* No packed fp32 arithmetic.
* No scratch memory and no spilled registers, but in the backward norm of rows
  whose width is not a multiple of 8, known to spill a few.
* The products' loads into LDS are written as asm, whose inside the compiler does
  not look at.  A scalar register that a vector instruction wrote needs five
  wait states before a memory instruction reads it, and M0 one: nothing in front
  of such a load may break that.
* The matrix instructions are there, and the streaming kernels load 16 bytes at
  a time.
"""

import os
import re
import shutil

import pytest

from swiglu_backward_int8_amd import _build

pytestmark = pytest.mark.skipif(not os.path.exists(_build.hipcc()) and shutil.which("hipcc") is None,
                                reason="hipcc is not installed")

SRC = [os.path.join(_build.PKG, "csrc", n + ".hip") for n in ("rmsnorm", "mxfp4", "mxfp4gemm")]


@pytest.fixture(scope="module")
def asm():
    return {os.path.basename(s)[:-4]: _build.device_asm(s) for s in SRC}


def kernels(text):
    """kernel symbol -> its lines, labels included, to the end of the function."""
    out = {}
    for m in re.finditer(r"^(_Z\S+):", text, re.M):
        end = text.find(".Lfunc_end", m.end())
        lines = [l.strip() for l in text[m.end():end].splitlines()]
        out[m.group(1)] = [l for l in lines if l and not l.startswith((";", "//")) and (not l.startswith(".") or l.endswith(":"))]
    return {k: v for k, v in out.items() if any(l.startswith("s_endpgm") for l in v)}


def metadata(text):
    meta = {}
    for m in re.finditer(r"\.name:\s+(\S+)(.*?)(?=\n\s+- \.|\n\s*\.end_amdgpu_metadata)", text, re.S):
        get = lambda key: int(re.search(r"\." + key + r":\s+(\d+)", m.group(2)).group(1))
        meta[m.group(1)] = (get("private_segment_fixed_size"), get("vgpr_spill_count"))
    return meta


def test_no_packed_fp32(asm):
    packed = re.compile(r"\bv_pk_(fma|mul|add)_f32\b")
    for name, text in asm.items():
        assert kernels(text)
        assert not packed.search(text), name


def test_no_spills(asm):
    for text in asm.values():
        for name, (scratch, spills) in metadata(text).items():
            if "rms_norm_bwd_kernelILb0E" in name and "KindE2" in name:
                assert scratch <= 64, (name, scratch)
            else:
                assert scratch == 0 and spills == 0, (name, scratch, spills)


def registers(operand):
    m = re.match(r"s\[(\d+):(\d+)\]$", operand)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    m = re.match(r"s(\d+)$", operand)
    return {int(m.group(1))} if m else {"m0"} if operand == "m0" else set()


def hazards(lines):
    """Loads into LDS that come too soon after a write of their scalars, and how many there were."""
    bad, seen, back = [], 0, []
    for line in lines:
        if line.endswith(":"):
            continue  # what falls through a label still counts
        op, *rest = line.split(None, 1)
        args = [a.strip() for a in rest[0].split(",")] if rest else []
        if "lds" in line.split() and op.startswith("buffer_load"):
            seen += 1
            reads = set().union(*(registers(a.split()[0]) for a in args[1:] if a))
            states = 0
            for p, pargs in reversed(back):
                if states >= 5:
                    break
                writes = registers(pargs[0]) if pargs and p.startswith(("v_read", "v_cmp", "s_mov", "s_add", "v_add_co")) else set()
                if p.startswith("v_") and writes & reads or ("m0" in writes and states < 1):
                    bad.append((p, pargs, line))
                states += int(pargs[0]) + 1 if p == "s_nop" else 1
        back.append((op, args))
        back = back[-6:]
    return bad, seen


def test_loads_into_lds_wait_for_their_scalars(asm):
    total = 0
    for name, lines in kernels(asm["mxfp4gemm"]).items():
        bad, seen = hazards(lines)
        assert not bad, (name, bad[:3])
        total += seen
    assert total > 100


def test_the_hazard_check_sees_hazards():
    load = "buffer_load_dwordx4 v1, s[4:7], s9 offen lds"
    assert not hazards(["v_readlane_b32 s3, v9, 1", "s_nop 0", load])[0]
    assert hazards(["v_readlane_b32 s6, v9, 1", "s_nop 0", load])[0]
    assert not hazards(["v_readlane_b32 s6, v9, 1", "s_nop 4", load])[0]
    assert hazards(["v_readfirstlane_b32 s9, v9", "s_nop 2", load])[0]
    assert hazards(["s_mov_b32 m0, s2", load])[0]
    assert not hazards(["s_mov_b32 m0, s2", "s_nop 0", load])[0]


def test_instructions(asm):
    for name, lines in kernels(asm["mxfp4gemm"]).items():
        body = "\n".join(lines)
        assert "v_mfma_scale_f32_" in body, name
        if "stream" not in name:
            assert "v_mfma_scale_f32_32x32x64_f8f6f4" in body and "buffer_load_dwordx4" in body, name
    for src, kernel in (("rmsnorm", "rms_norm_quant_kernel"), ("mxfp4", "MxQuantRows"), ("mxfp4", "mx_quant_both")):
        found = [l for n, l in kernels(asm[src]).items() if kernel in n and "KindE3" not in n]
        assert found and all(any(x.startswith("global_load_dwordx4") for x in l) for l in found), kernel
    both = [l for n, l in kernels(asm["mxfp4"]).items() if "mx_quant_both" in n]
    assert all(any(x.startswith("v_cvt_scalef32_pk_fp4_bf16") for x in l) for l in both)
