"""Sizes T, H, D of the gated projection for the kernels that other tests' sizes leave
out, and the product and the tiles that each is for: rows, columns and K that these
tiles do not divide."""

# 8 slices of K where it says so
ONE_TILE_EACH = {
    (782, 4432, 1168): ("dx", "k256", 8),
    (3390, 72, 2320): ("dx", "k256", 1),
    (16495, 40, 152): ("dx", "k128Two", 1),
    (8124, 328, 1304): ("dw", "k256", 8),
    (129, 1168, 3368): ("dw", "k256", 1),
}
SHAPES = list(ONE_TILE_EACH)
