"""Sizes that the GPU tests mean for one form of the 8-bit products' kernels, and that form.

A size is (rows of x, rows sharing one, groups (0: no tables), contracted elements, output columns); a form is
the output rows, output columns and wavefronts of a workgroup and the stages that it holds (0: streaming).
Each tiled form gets contracted dimensions that are and that are not multiples of 128, of fewer stages than a
round of its loop and of more; test_block_forms.py checks that each size takes its form."""

STREAM_DEEP, STREAM_WIDE = (32, 16, 8, 0), (32, 32, 4, 0)
TILE_64_8, TILE_64_4 = (64, 64, 4, 8), (64, 64, 4, 4)
TILE_128_4, TILE_128_2, TILE_256 = (128, 128, 4, 4), (128, 128, 4, 2), (256, 256, 8, 2)

FORWARD = {
    STREAM_DEEP: [(3, 1, 0, 144, 272), (45, 2, 2, 1168, 144), (24, 1, 3, 4368, 400), (33, 1, 0, 1280, 1040)],
    STREAM_WIDE: [(9, 1, 0, 144, 8208), (45, 2, 130, 400, 144), (24, 1, 7, 1680, 1040), (150, 1, 7, 1280, 2064)],
    TILE_64_8: [(777, 2, 2, 656, 272), (777, 2, 0, 1280, 528), (333, 1, 3, 1168, 2064), (1300, 2, 0, 384, 272)],
    TILE_64_4: [(80, 2, 2, 400, 8208), (80, 2, 3, 384, 8208), (1111, 1, 0, 656, 2064), (2050, 1, 0, 640, 1040)],
    TILE_128_4: [(1300, 2, 2, 144, 1040), (1300, 2, 0, 384, 1040), (1111, 1, 7, 656, 2064), (600, 1, 3, 640, 4112)],
    TILE_128_2: [(777, 2, 7, 144, 2064), (210, 2, 0, 384, 8208), (333, 1, 3, 656, 8208), (2050, 1, 0, 640, 2064)],
    TILE_256: [(777, 2, 7, 144, 4112), (777, 2, 7, 384, 4112), (1111, 1, 0, 656, 8208), (2050, 1, 0, 640, 4112)],
}
DX = {
    TILE_64_8: [(3, 1, 0, 144, 272), (45, 2, 2, 1168, 144), (24, 1, 3, 1280, 400), (333, 1, 3, 1168, 2064)],
    TILE_64_4: [(45, 2, 130, 144, 144), (45, 2, 0, 384, 8208), (1111, 1, 0, 656, 2064), (2050, 1, 0, 640, 1040)],
    TILE_128_4: [(1300, 2, 2, 144, 1040), (1300, 2, 0, 384, 1040), (1111, 1, 7, 656, 2064), (600, 1, 3, 640, 4112)],
    TILE_128_2: [(777, 2, 7, 144, 2064), (210, 2, 0, 384, 8208), (333, 1, 3, 656, 8208), (2050, 1, 0, 640, 2064)],
    TILE_256: [(777, 2, 7, 144, 4112), (777, 2, 7, 384, 4112), (1111, 1, 0, 656, 8208), (2050, 1, 0, 640, 4112)],
}


def cases():
    """(dx, size, form) of all of them."""
    for dx, sizes in ((False, FORWARD), (True, DX)):
        for form, of in sizes.items():
            for size in of:
                yield dx, size, form
