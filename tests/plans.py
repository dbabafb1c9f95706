"""Which kernels the gated projection takes at a size: csrc/swiglu_plan.h, compiled for
the CPU."""

import functools
import os
import subprocess
import tempfile

from swiglu_backward_int8_amd import _build

TILES = ("k256", "k128", "k128Two", "k64")
SHAPE = {"k256": (256, 256), "k128": (128, 128), "k128Two": (128, 128), "k64": (64, 128)}  # rows of A and of B

PROGRAM = r"""
#include <stdio.h>
#include "swiglu_plan.h"
int main() {
  long long T, H, D;
  while (scanf("%lld %lld %lld", &T, &H, &D) == 3) {
    const swiglu::Plan f = swiglu::plan(T, 2 * H, D, false, false), x = swiglu::plan(T, D, 2 * H, false, true),
                       w = swiglu::plan(2 * H, D, T, true, true);
    printf("%d %d %d %d %d %d\n", swiglu::streamed(T, H, D), f.tiles, x.tiles, x.slices, w.tiles, w.slices);
  }
}
"""


@functools.lru_cache(None)
def _program():
    folder = tempfile.mkdtemp()
    source, program = os.path.join(folder, "p.cpp"), os.path.join(folder, "p")
    with open(source, "w") as f:
        f.write(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I" + os.path.join(_build.PKG, "csrc"), source, "-o", program], check=True)
    return program


def kernels(shapes):
    """For each (T, H, D) the kernels of its three products: ("gated", "stream", blocks of
    16 rows) or (product, tiles, slices)."""
    out = subprocess.run([_program()], input="".join("%d %d %d\n" % s for s in shapes), capture_output=True, text=True, check=True)
    found = []
    for (T, H, D), line in zip(shapes, out.stdout.splitlines()):
        blocks, f, x, xs, w, ws = map(int, line.split())
        gated = ("gated", "stream", blocks) if blocks else ("gated", TILES[f], 1)
        found.append((gated, ("dx", TILES[x], xs), ("dw", TILES[w], ws)))
    assert len(found) == len(shapes)
    return found
