"""Shapes of the experts' product over a plan with replica slots, at least two for the forms that
many rows take and one for every other, with the form that the library chooses for the plain
product and for SwiGLU: channels, rows and depths that end inside a tile, a block of 16 and a step."""

# rows, R, E, S, N, D, form plain, form SwiGLU
SHAPES = [
    (3001, 4, 12, 1, 1040, 144, "large", "large"),
    (2000, 2, 6, 1, 2064, 272, "large", "large"),
    (2304, 4, 28, 1, 1040, 1040, "128x128", "128x128"),
    (2304, 1, 32, 0, 4112, 528, "128x128", "128x128"),
    (1037, 2, 6, 1, 4112, 400, "128x128", "128x128"),
    (1108, 4, 8, 1, 2096, 864, "128x128 deep", "128x128 deep"),
    (1000, 2, 2, 1, 1040, 4112, "64x128", "64x128"),
    (1100, 4, 16, 1, 2064, 528, "128x64", "128x64"),
    (240, 1, 1, 1, 3168, 336, "64x64", "64x64"),
    (69, 4, 12, 1, 944, 432, "64x32 deep", "64x32 deep"),
    (60, 4, 16, 1, 2064, 528, "64x32", "64x32"),
    (50, 2, 2, 1, 2064, 272, "32x32", "32x32"),
    (20, 1, 1, 1, 2064, 4112, "32x16", "32x16"),
    (12, 2, 2, 1, 528, 2064, "16x16", "32x16"),
]
