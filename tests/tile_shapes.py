"""Sizes T, H, D of the gated projection for the kernels that other tests' sizes leave
out, and the product and the tiles that each is for: rows, columns and K that these
tiles do not divide."""

# one tile a workgroup; 8 slices of K where it says so
ONE_TILE_EACH = {
    (782, 4432, 1168): ("dx", "k256", 8),
    (3390, 72, 2320): ("dx", "k256", 1),
    (16495, 40, 152): ("dx", "k128Two", 1),
    (8124, 328, 1304): ("dw", "k256", 8),
    (129, 1168, 3368): ("dw", "k256", 1),
}
# workgroups that take several tiles, whole ones behind partial ones and the other way round
SEVERAL_TILES = {
    (3501, 3512, 216): ("gated", "k256", 1),
    (9001, 6008, 200): ("gated", "k256", 1),     # up to seven each
    (2632, 3096, 592): ("gated", "k128", 1),
    (286, 10896, 72): ("gated", "k128Two", 1),
    (165, 10744, 856): ("gated", "k64", 1),
    (7863, 104, 3080): ("dx", "k256", 1),
    (9003, 520, 9224): ("dx", "k256", 1),        # up to six each
    (4267, 304, 3864): ("dx", "k128", 1),
    (21972, 40, 280): ("dx", "k128Two", 1),
    (445, 1032, 9120): ("dx", "k64", 1),
    (195, 4448, 2736): ("dw", "k256", 1),
    (1030, 9224, 9000): ("dw", "k256", 1),       # up to eleven each
    (614, 2376, 3408): ("dw", "k128", 1),
    (65, 11616, 280): ("dw", "k128Two", 1),
}
SHAPES = list(ONE_TILE_EACH) + list(SEVERAL_TILES)
