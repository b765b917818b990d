"""Launches of the FP4 x FP4 GEMMs stay below 2^32 threads at the borders of what the entry points take (CPU: the plan and the
bound of row tiles run on the host)."""
import ctypes
import os
import random

import pytest

import block_scaled_fp8_dispatch_amd as moe
from fp4_kernel_cases import plan

pytestmark = pytest.mark.skipif(not os.path.exists(moe.LIB_PATH), reason="library not built")

# rows of the row tiles, rows and columns of a workgroup's output, its threads
FORM = {"tiled 256": (256, 256, 256, 256), "tiled 128": (128, 128, 256, 256), "tiled 64": (64, 64, 256, 256),
        "skinny 64x64": (64, 64, 64, 512), "skinny 32x64": (64, 32, 64, 512), "skinny 32x32": (64, 32, 32, 512),
        "skinny 16x32": (64, 16, 32, 512), "skinny 16": (64, 16, 16, 1024)}


def most_row_tiles(rows, groups, block_m):
    f = moe.load_library()._ZN3moe14most_row_tilesEiii
    f.argtypes, f.restype = [ctypes.c_int] * 3, ctypes.c_int
    return f(rows, groups, block_m)


def threads(layout, M, G, N, kernel):
    """Of the product's launch: a workgroup for each tile that the lists or counts can name, columns in whole fragments of 128 for
    the skinny kernels, and the workgroups that a last round of 256-row tiles may take more."""
    block_m, bm, bn, t = FORM[kernel]
    if layout == "dense":
        units = -(-M // (bm if kernel.startswith("skinny") else block_m))
    elif layout == "contiguous":
        units = most_row_tiles(M, G, block_m) * (block_m // bm)
    else:
        units = G * -(-M // block_m) * (block_m // bm)
    columns = -(-N // 128) * (128 // bn) if kernel.startswith("skinny") else -(-N // 256)
    return (units * columns + (256 if kernel == "tiled 256" else 0)) * t


@pytest.mark.parametrize("block_m", [64, 128, 256])
def test_row_tiles_of_groups(block_m):
    """The bound holds for every split of rows into groups, and some split reaches it."""
    rng = random.Random(block_m)
    for _ in range(2000):
        groups = rng.choice((1, 2, 3, 7, 64, 1024))
        rows = [rng.choice((0, 1, block_m - 1, block_m, block_m + 1, rng.randrange(5 * block_m))) for _ in range(groups)]
        most = most_row_tiles(sum(rows), groups, block_m)
        assert sum(-(-r // block_m) for r in rows) <= most
        # a masked product's groups all have the same capacity
        assert groups * -(-rows[0] // block_m) <= most_row_tiles(groups * rows[0], groups, block_m)
    for groups in (2, 5, 63):
        rows = [1] * (groups - 1) + [3 * block_m + 1]
        assert sum(-(-r // block_m) for r in rows) == groups + 3 == most_row_tiles(sum(rows), groups, block_m)
    assert most_row_tiles(2 ** 31 - 1 - 1024 * 256, 1024, block_m) > 0


def accepted(rows, G, N, K):
    return N <= 2 ** 30 and rows * K < 2 ** 32 and most_row_tiles(rows, G, 128) * -(-N // 256) < 2 ** 24


def test_largest_launches():
    """Just inside the refusal: groups and rows of all sizes, the most columns that are still taken."""
    border = 0
    for K in (128, 512, 7168):
        for G in (1, 2, 4, 7, 64, 65, 1000, 1024):
            for M in (1, 2, 33, 64, 65, 127, 128, 129, 255, 256, 257, 1000, 4097, 65535, 2 ** 20 + 1):
                for layout in ("dense", "contiguous", "masked"):
                    if layout == "dense" and G > 1:
                        continue
                    rows = G * M if layout == "masked" else M
                    tiles = (2 ** 24 - 1) // most_row_tiles(rows, G, 128)
                    for N in {min(2 ** 30, 256 * tiles), min(2 ** 30, 256 * tiles - 240), 256 * (tiles // 2), 256 * (tiles // 17) + 16, 128 * tiles + 16}:
                        if N < 16 or not accepted(rows, G, N, K):
                            continue
                        border += 1
                        kernel, _ = plan(layout, M, G, N, K, M)
                        assert threads(layout, M, G, N, kernel) < 2 ** 32, (layout, M, G, N, K, kernel)
    assert border > 3000
