"""Sizes that the GPU tests mean for one form of the kernels, and that form.

A size is (rows of x, rows sharing one, groups (0: no tables), h_in, h_out); a form is the output
rows, output columns and wavefronts of a workgroup.  test_kernel_forms.py checks that each size
takes its form, so that a change of the rules cannot leave a kernel without its tests."""

STREAM_16 = (32, 16, 4)
STREAM_4_WIDE, STREAM_4_DEEP = (32, 32, 2), (32, 16, 8)
TILE_128, TILE_HALF, TILE_256 = (128, 128, 4), (128, 256, 4), (256, 256, 8)

# 16-bit weights, streamed: dense and grouped, groups of up to 16, up to 32 and more rows, h_in and
# h_out that end inside a unit and a column tile
STREAMED = [
    (1, 1, 0, 1032, 264), (3, 1, 0, 2056, 136), (16, 1, 0, 1032, 8), (17, 1, 0, 1096, 72), (32, 1, 0, 2048, 64),
    (33, 1, 0, 4104, 264), (40, 1, 0, 4104, 264), (1, 2, 5, 1032, 264), (12, 2, 4, 1160, 136),
    (45, 2, 3, 2056, 264), (300, 1, 130, 2056, 72), (100, 2, 2, 2184, 40), (3, 4, 64, 1160, 24),
]
# the same where rows of one size do for a test of its own
STREAMED_FAR = (5, 1, 2, 1096, 136)
STREAMED_MIXED = [(24, 1, 4, 1160, 136), (150, 1, 4, 2056, 136)]
STREAMED_REPEATED = [(20, 2, 6, 1544, 264)]

# 4-bit weights, streamed: 8 wavefronts, or 2 of them over 32 columns
MX_DEEP = [(4, 1, 3, 2080, 72), (60, 1, 3, 2080, 72), (20, 2, 5, 2336, 264), (1, 1, 0, 2080, 264),
           (24, 1, 0, 2304, 264)]
MX_WIDE = [(8, 1, 3, 2080, 3000), (60, 1, 3, 2080, 3000), (5, 1, 0, 2080, 8200), (24, 1, 0, 2304, 8200)]
# and in tiles, 16-bit rows
MX_TILES = {TILE_128: [(300, 1, 0, 160, 264)], TILE_HALF: [(1100, 1, 0, 160, 7000)],
            TILE_256: [(4096, 1, 0, 160, 4096), (3600, 1, 2, 96, 4088), (3600, 1, 2, 544, 4088)]}
# both sides in 4 bits: streamed only where few rows meet long weights (15 rows to a group on
# average are more than 16 in many)
BOTH_DEEP = [(4, 1, 3, 8224, 72), (60, 1, 3, 8224, 72), (20, 2, 5, 8416, 264), (1, 1, 0, 4128, 264),
             (24, 1, 0, 8416, 264)]
BOTH_WIDE = [(300, 1, 20, 6176, 296), (5, 1, 0, 5152, 8200)]
BOTH_TILES = {TILE_128: [(300, 1, 0, 160, 264)], TILE_256: [(4096, 1, 0, 160, 4096)]}


def cases():
    """(mode, size, form) of all of them; modes as in the kernels' own list."""
    forward, mx, both = "forward", "mx", "both"
    for size in [*STREAMED, STREAMED_FAR, *STREAMED_MIXED, *STREAMED_REPEATED]:
        yield forward, size, STREAM_16
    for mode, deep, wide in ((mx, MX_DEEP, MX_WIDE), (both, BOTH_DEEP, BOTH_WIDE)):
        for size in deep:
            yield mode, size, STREAM_4_DEEP
        for size in wide:
            yield mode, size, STREAM_4_WIDE
    for mode, tiles in ((mx, MX_TILES), (both, BOTH_TILES)):
        for form, sizes in tiles.items():
            for size in sizes:
                yield mode, size, form
