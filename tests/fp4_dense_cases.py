"""Dense products that the FP4 x FP4 GEMMs' cost model sends to each kernel's two forms: B read past the caches, as up to one row tile
of rows does (64, 128 or 256 of them), or not. M, N, K, kernel, past the caches. (The 256-row kernel has one form.)"""

CASES = [
    (129, 21856, 256, "tiled 256", True), (2100, 2608, 1536, "tiled 256", False),
    (65, 32944, 256, "tiled 128", True), (127, 32944, 128, "tiled 128", True), (258, 16416, 128, "tiled 128", False),
    (60, 34960, 256, "tiled 64", True), (33, 18160, 896, "tiled 64", True), (30, 34960, 512, "tiled 64", True),
    (100, 8416, 640, "tiled 64", False), (65, 16144, 512, "tiled 64", False),
    (33, 8752, 2048, "skinny 64x64", True), (100, 4384, 2048, "skinny 64x64", False),
    (19, 13792, 2048, "skinny 32x64", True), (129, 2032, 2048, "skinny 32x64", False),
    (24, 8752, 2560, "skinny 32x32", True), (21, 22192, 1152, "skinny 32x32", True), (127, 4720, 896, "skinny 32x32", False),
    (3, 34960, 5120, "skinny 16x32", True), (14, 33280, 1152, "skinny 16x32", True), (1, 16, 128, "skinny 16x32", True),
    (69, 3040, 2560, "skinny 16x32", False),
    (1, 16, 2560, "skinny 16", True), (64, 1024, 7168, "skinny 16", True), (69, 688, 7168, "skinny 16", False),
]
