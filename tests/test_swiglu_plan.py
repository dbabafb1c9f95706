"""The sizes of the gated projection's GPU tests reach every kernel that its planner
can choose: each product, with each of its tiles, in one piece and in slices of K, with
one and with several tiles a workgroup (CPU only)."""

import random

import pytest

import plans
import test_swiglu_gemm_gpu as gemm
import tile_shapes


def kind(kernel):
    """Slices as whether there are any: their number is a dimension of the grid."""
    return kernel if kernel[1] == "stream" else (kernel[0], kernel[1], kernel[2] > 1, kernel[3])


def kinds(shapes):
    return {kind(k) for found in plans.kernels(shapes) for k in found}


def drawn(n):
    r = random.Random(11)
    whole = lambda low, high: max(8, int(2 ** r.uniform(low, high)) // 8 * 8)
    return [(int(2 ** r.uniform(0, 20)), whole(3, 17), whole(3, 17)) for _ in range(n)]


def test_every_kernel_is_reached():
    tested = kinds(gemm.SHAPES + tile_shapes.SHAPES)
    can_be = kinds(drawn(100000))
    assert len(can_be) == 3 + 4 * 2 + 4 * 3 + 3 * 3  # streams; gated, dx and dw tiles: one, several, (but gated) sliced
    assert tested == can_be


def test_every_number_of_slices_is_reached():
    of = lambda shapes: {(k[0], k[2]) for found in plans.kernels(shapes) for k in found if k[0] != "gated"}
    assert of(gemm.SHAPES + tile_shapes.SHAPES) >= {(p, n) for p in ("dx", "dw") for n in (1, 2, 4, 8, 16)}


def sizes(product, T, H, D):
    """Rows, columns and K of a product."""
    return {"gated": (T, 2 * H, D), "dx": (T, D, 2 * H), "dw": (2 * H, D, T)}[product]


@pytest.mark.parametrize("shape", tile_shapes.SHAPES)
def test_shapes_are_for_what_they_say(shape):
    several = shape in tile_shapes.SEVERAL_TILES
    product, tiles, slices = (tile_shapes.SEVERAL_TILES if several else tile_shapes.ONE_TILE_EACH)[shape]
    assert (product, tiles, slices, several) in plans.kernels([shape])[0]
    M, columns, K = sizes(product, *shape)
    a, b = plans.SHAPE[tiles]
    assert M > a and columns > b and M % a != 0 and columns % b != 0 and K % 64 != 0
    turns = plans.sequences(tiles, M, columns)
    m, n = plans.tile_counts(tiles, M, columns)
    assert sum(map(len, turns)) == m * n
    pairs = {p for t in turns for p in zip(t, t[1:])}
    assert {(True, True), (True, False), (False, True)} <= pairs if several else not pairs
