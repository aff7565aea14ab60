"""Sizes that take each of the linear layer's kernels: (m, n, K, weights, gated,
MXFP8 output). The host test evaluates the choice of kernel for each; the GPU
test compares their values with the definition."""

# Few rows, scaled products: 16 columns and 8 waves, 32 and 8 (MXFP8 output), 32
# and 4 (more than 8192 columns; gated with an MXFP8 output), each for up to 16
# rows and for more.
FEW = [
    (5, 300, 1056, "MXFP4", False, False), (20, 1000, 544, "MXFP8", False, False),
    (16, 250, 288, "MXFP8", True, False), (40, 500, 160, "MXFP4", True, False),
    (16, 4096, 544, "MXFP4", False, True), (9, 4096, 288, "MXFP8", False, True),
    (24, 4096, 544, "MXFP4", False, True), (17, 2048, 288, "MXFP8", False, True),
    (1, 14336, 1024, "MXFP4", False, False), (2, 14336, 1056, "MXFP8", False, False),
    (20, 9000, 544, "MXFP4", False, False), (20, 9000, 288, "MXFP8", False, False),
    (3, 14336, 288, "MXFP4", False, True), (20, 9216, 288, "MXFP8", False, True),
    (1, 14336, 544, "MXFP4", True, False), (20, 9001, 288, "MXFP8", True, False),
    (9, 4096, 544, "MXFP4", True, True), (17, 2080, 288, "MXFP8", True, True),
    (4, 9216, 288, "MXFP8", True, True), (20, 9216, 160, "MXFP4", True, True),
]

# (rows of a tile, K parts) and sizes: scales read as they stand (K a multiple of
# 512; never in tiles of 256 rows) and in another order.
TILES = [
    ((32, 1), [(33, 14336, 512, "MXFP4", False, False), (33, 14336, 512, "MXFP8", False, True),
               (12, 14336, 1024, "MXFP4", True, False), (12, 14336, 512, "MXFP8", True, True),
               (129, 5410, 1056, "MXFP4", False, False), (129, 5410, 1056, "MXFP8", False, False),
               (40, 8192, 2080, "MXFP4", True, True), (12, 14336, 2080, "MXFP8", True, False),
               (24, 14336, 4096, "MXFP4", True, True), (333, 2050, 2080, "MXFP8", False, False)]),
    ((32, 2), [(12, 64, 8192, "MXFP4", False, False), (33, 1024, 4096, "MXFP8", False, True),
               (700, 64, 2048, "MXFP4", True, True), (12, 64, 4096, "MXFP8", True, False),
               (12, 4096, 14336, "MXFP4", False, True), (257, 1000, 4128, "MXFP8", False, False),
               (300, 1000, 4128, "MXFP4", False, False), (24, 14336, 4128, "MXFP8", False, True),
               (24, 1824, 4128, "MXFP4", True, True), (33, 1024, 4128, "MXFP8", True, True)]),
    ((64, 1), [(129, 7000, 512, "MXFP4", False, False), (500, 2080, 512, "MXFP8", False, True),
               (257, 1824, 512, "MXFP4", True, True), (100, 4160, 512, "MXFP8", True, False),
               (500, 4096, 288, "MXFP4", False, False), (90, 14336, 544, "MXFP8", False, True),
               (33, 14336, 1056, "MXFP4", True, True), (100, 8192, 544, "MXFP8", True, False)]),
    ((64, 2), [(700, 64, 8192, "MXFP4", False, True), (700, 64, 8192, "MXFP8", False, False),
               (33, 1824, 4096, "MXFP4", True, True), (257, 96, 8192, "MXFP8", True, False),
               (257, 1824, 4128, "MXFP4", False, True), (33, 7000, 4128, "MXFP8", False, False),
               (50, 5410, 4128, "MXFP4", True, False), (33, 1824, 4128, "MXFP8", True, True)]),
    ((128, 1), [(257, 7000, 512, "MXFP4", False, False), (129, 14336, 512, "MXFP8", False, True),
                (200, 4160, 512, "MXFP4", True, True), (200, 4160, 512, "MXFP8", True, False),
                (200, 14336, 256, "MXFP4", False, True), (129, 14336, 288, "MXFP8", False, False),
                (333, 5410, 288, "MXFP4", True, False), (100, 14336, 256, "MXFP8", True, True)]),
    ((128, 2), [(1500, 64, 14336, "MXFP4", False, True), (1100, 64, 8192, "MXFP8", False, False),
                (90, 2050, 8192, "MXFP4", True, False), (90, 2080, 4096, "MXFP8", True, True),
                (90, 5410, 4128, "MXFP8", False, False), (129, 1824, 4128, "MXFP8", True, True)]),
    ((256, 1), [(257, 14336, 256, "MXFP4", False, True), (257, 14336, 256, "MXFP8", False, False),
                (333, 8192, 256, "MXFP4", True, True), (129, 14336, 256, "MXFP8", True, False)]),
    ((256, 2), [(257, 14336, 8192, "MXFP4", False, False), (129, 5410, 14336, "MXFP8", False, False),
                (257, 14336, 4128, "MXFP8", False, True), (200, 4160, 14336, "MXFP4", True, True),
                (257, 1824, 14336, "MXFP8", True, False)]),
]


def all_cases():
    return FEW + [c for _, cases in TILES for c in cases]


def name(c):
    return f"{c[0]}x{c[1]}{'gated' if c[4] else ''}x{c[2]}-{c[3]}-{'mx8' if c[5] else 'bf16'}"
