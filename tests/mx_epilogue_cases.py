"""Sizes of the GPU tests of products with an epilogue and of experts' products, and the tiles that each is there for."""

# rows, columns, depth, groups -> tile (0: the kernel of few rows; 96: 64 x 128)
GROUPED_TILES = {
    (1, 40, 64, 1): 0, (16, 100, 320, 70): 0, (7, 33, 1000, 3): 0,
    (17, 64, 96, 2): 64, (200, 1024, 544, 8): 64, (33, 130, 2050, 5): 64,
    (520, 1500, 300, 64): 96, (301, 1030, 257, 100): 96,
    (2000, 2570, 520, 5): 128, (4100, 4100, 1030, 8): 128,
    (8111, 4097, 3300, 2): 128, (6101, 4099, 4130, 2): 256, (7300, 4100, 4352, 2): 256,
}
# rows, M, N, groups -> tile
GRADIENT_TILES = {(300, 130, 200, 3): 128, (5, 66, 40, 2): 128, (3000, 1030, 544, 3): 128, (300, 4099, 2570, 9): 256,
                  (260, 4096, 2560, 6): 256}
