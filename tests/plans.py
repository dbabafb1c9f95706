"""Which kernels the gated projection takes at a size: csrc/swiglu_plan.h, compiled for
the CPU, and the order in which a workgroup takes its tiles."""

import functools
import os
import subprocess
import tempfile

from swiglu_backward_int8_amd import _build

TILES = ("k256", "k128", "k128Two", "k64")
SHAPE = {"k256": (256, 256), "k128": (128, 128), "k128Two": (128, 128), "k64": (64, 128)}  # rows of A and of B
PER_CU = {"k256": 1, "k128": 1, "k128Two": 2, "k64": 1}
XCDS, CUS_OF_XCD, RASTER_ROWS = 8, 32, 4

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


def tile_counts(tiles, M, columns):
    a, b = SHAPE[tiles]
    return -(-M // a), -(-columns // b)


def several(tiles, M, columns):
    """Whether some workgroup takes more than one tile of a product (of one slice)."""
    m, n = tile_counts(tiles, M, columns)
    return -(-m * n // XCDS) > CUS_OF_XCD * PER_CU[tiles]


def kernels(shapes):
    """For each (T, H, D) the kernels of its three products: ("gated", "stream", blocks of
    16 rows) or (product, tiles, slices, whether a workgroup takes several tiles)."""
    out = subprocess.run([_program()], input="".join("%d %d %d\n" % s for s in shapes), capture_output=True, text=True, check=True)
    found = []
    for (T, H, D), line in zip(shapes, out.stdout.splitlines()):
        blocks, f, x, xs, w, ws = map(int, line.split())
        gated = ("gated", "stream", blocks) if blocks else ("gated", TILES[f], 1, several(TILES[f], T, 2 * H))
        found.append((gated, ("dx", TILES[x], xs, several(TILES[x], T, D)), ("dw", TILES[w], ws, several(TILES[w], 2 * H, D))))
    assert len(found) == len(shapes)
    return found


def sequences(tiles, M, columns):
    """For each workgroup of a product: for its tiles in turn, whether the tile is whole."""
    a, b = SHAPE[tiles]
    m, n = tile_counts(tiles, M, columns)
    per_xcd = -(-m * n // XCDS)
    slots = min(per_xcd, CUS_OF_XCD * PER_CU[tiles])
    out = []
    for xcd in range(XCDS):
        end = min((xcd + 1) * per_xcd, m * n)
        for slot in range(slots):
            turn = []
            for at in range(xcd * per_xcd + slot, end, slots):
                group, inside = divmod(at, RASTER_ROWS * n)
                rows = min(m - RASTER_ROWS * group, RASTER_ROWS)
                column, row = divmod(inside, rows)
                row += RASTER_ROWS * group
                turn.append((row + 1) * a <= M and (column + 1) * b <= columns)
            out.append(turn)
    return out
