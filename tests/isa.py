"""gfx950 assembly of the sources, for the checks of the instructions: kernels as
instructions with the paths between them (every source is compiled once a run)."""

import functools
import os
import re

from swiglu_backward_int8_amd import _build

OPERATORS = ("rmsnorm", "mxfp4", "mxfp4gemm")


@functools.lru_cache(None)
def text(source):
    return _build.device_asm(os.path.join(_build.PKG, "csrc", source + ".hip"))


class Kernel:
    """Instructions (mnemonic, operands) in order, and where control can come from."""

    def __init__(self, lines):
        self.code, labels = [], {}
        for line in lines:
            line = re.sub(r"(;|//).*", "", line).strip()
            if line.endswith(":"):
                labels[line[:-1]] = len(self.code)
            elif line and not line.startswith("."):
                op, *rest = line.split(None, 1)
                self.code.append((op, [a.strip() for a in rest[0].split(",")] if rest else []))
        self.before = [[] for _ in self.code]  # the instructions that can come right before each
        for i, (op, args) in enumerate(self.code):
            if op in ("s_branch",) or op.startswith("s_cbranch"):
                to = labels[args[0]]
                if to < len(self.code):
                    self.before[to].append(i)
            if op not in ("s_branch", "s_endpgm") and i + 1 < len(self.code):
                self.before[i + 1].append(i)
        self.targets = set(labels.values())

    def blocks(self):
        """Runs of instructions that nothing enters or leaves but at their ends."""
        start = 0
        for i, (op, _) in enumerate(self.code):
            if i in self.targets and i > start:
                yield self.code[start:i]
                start = i
            if op == "s_branch" or op.startswith("s_cbranch") or op == "s_endpgm":
                yield self.code[start:i + 1]
                start = i + 1


@functools.lru_cache(None)
def kernels(source):
    """kernel symbol -> Kernel."""
    asm, out = text(source), {}
    for m in re.finditer(r"^(_Z\S+):", asm, re.M):
        lines = asm[m.end():asm.find(".Lfunc_end", m.end())].splitlines()
        if any(l.strip().startswith("s_endpgm") for l in lines):
            out[m.group(1)] = Kernel(lines)
    return out


def metadata(source):
    """kernel symbol -> (bytes of scratch, spilled vector registers, spilled scalar registers)."""
    out = {}
    for m in re.finditer(r"\.name:\s+(\S+)(.*?)(?=\n\s+- \.|\n\s*\.end_amdgpu_metadata)", text(source), re.S):
        get = lambda key: int(re.search(r"\." + key + r":\s+(\d+)", m.group(2)).group(1))
        out[m.group(1)] = (get("private_segment_fixed_size"), get("vgpr_spill_count"), get("sgpr_spill_count"))
    return out


def into_lds(op, args):
    """Whether an instruction loads from memory into LDS."""
    return op.startswith("buffer_load") and bool(args) and "lds" in args[-1].split()


def scalars(operand):
    """The scalar registers of an operand ('s[4:7]', 's9 offen', 'm0', 'vcc')."""
    m = re.match(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    m = re.match(r"s(\d+)\b", operand)
    return {int(m.group(1))} if m else {"m0"} if re.match(r"m0\b", operand) else set()


def written(op, args):
    """The scalar registers that an instruction writes: the first operand's, and the
    second's of the vector instructions that give a carry or a flag there."""
    if not args or op.startswith(("s_cmp", "s_bitcmp", "s_cbranch", "s_waitcnt", "s_nop", "s_barrier", "s_branch",
                                  "buffer_", "global_", "ds_", "scratch_", "flat_")):
        return set()
    out = scalars(args[0])
    if "_co_" in op or op.startswith(("v_div_scale", "v_mad_u64", "v_mad_i64")):
        out |= scalars(args[1])
    return out
