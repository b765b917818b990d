"""Products that the FP4 x FP4 GEMMs' cost model sends to each of their kernels, and a view of what it picks.

A case: layout, M (dense, contiguous: rows; masked: capacity of a group), groups, N, K, expected rows a group (masked), the
kernel, and whether one row tile a group reads B (always False for dense)."""
import ctypes

import block_scaled_fp8_dispatch_amd as moe

KERNELS = ("tiled 256", "tiled 128", "tiled 64", "skinny 64x64", "skinny 32x64", "skinny 32x32", "skinny 16x32", "skinny 16")

CASES = [
    ("dense", 1300, 1, 4160, 640, 0, "tiled 256", False),
    ("dense", 2100, 1, 2608, 1536, 0, "tiled 256", False),
    ("dense", 258, 1, 16416, 128, 0, "tiled 128", False),
    ("dense", 65, 1, 32816, 128, 0, "tiled 128", False),
    ("dense", 3100, 1, 368, 640, 0, "tiled 64", False),
    ("dense", 300, 1, 4272, 2560, 0, "tiled 64", False),
    ("dense", 2100, 1, 368, 4608, 0, "skinny 64x64", False),
    ("dense", 900, 1, 640, 40064, 0, "skinny 64x64", False),     # scales of more K steps than LDS holds at once
    ("dense", 128, 1, 2608, 3712, 0, "skinny 32x64", False),
    ("dense", 2600, 1, 112, 896, 0, "skinny 32x32", False),
    ("dense", 700, 1, 256, 128, 0, "skinny 16x32", False),
    ("dense", 300, 1, 16, 5120, 0, "skinny 16", False),
    ("contiguous", 3100, 3, 4272, 256, 0, "tiled 256", False),
    ("contiguous", 3100, 27, 4160, 256, 0, "tiled 256", True),
    ("contiguous", 2100, 10, 2608, 640, 0, "tiled 128", False),
    ("contiguous", 1000, 10, 4272, 640, 0, "tiled 128", True),
    ("contiguous", 300, 3, 4160, 640, 0, "tiled 64", False),
    ("contiguous", 1300, 5, 1552, 1536, 0, "tiled 64", False),
    ("contiguous", 100, 27, 1552, 896, 0, "tiled 64", True),
    ("contiguous", 100, 10, 2608, 2048, 0, "tiled 64", True),
    ("contiguous", 600, 3, 1040, 5120, 0, "skinny 64x64", False),
    ("contiguous", 33, 5, 4160, 3712, 0, "skinny 64x64", True),
    ("contiguous", 1000, 10, 256, 3712, 0, "skinny 32x64", False),
    ("contiguous", 1747, 66, 16, 5120, 0, "skinny 32x64", True),
    ("contiguous", 1300, 5, 528, 256, 0, "skinny 32x32", False),
    ("contiguous", 150, 10, 480, 1152, 0, "skinny 32x32", True),
    ("contiguous", 1000, 10, 48, 896, 0, "skinny 16x32", False),
    ("contiguous", 16, 3, 368, 896, 0, "skinny 16x32", True),
    ("contiguous", 300, 3, 48, 4608, 0, "skinny 16", False),
    ("contiguous", 16, 3, 112, 5120, 0, "skinny 16", True),
    # masked, up to 64 groups and more (which are listed by a launch before)
    ("masked", 700, 10, 4160, 128, 700, "tiled 256", False),
    ("masked", 300, 27, 4272, 128, 151, "tiled 256", True),
    ("masked", 600, 10, 2608, 256, 201, "tiled 128", False),
    ("masked", 100, 27, 2080, 640, 51, "tiled 128", True),
    ("masked", 500, 66, 368, 256, 500, "tiled 128", False),
    ("masked", 128, 66, 1552, 256, 128, "tiled 128", True),
    ("masked", 700, 5, 896, 384, 700, "tiled 64", False),
    ("masked", 600, 27, 48, 5120, 600, "tiled 64", False),
    ("masked", 600, 27, 368, 128, 1, "tiled 64", True),
    ("masked", 33, 27, 1040, 2560, 33, "tiled 64", True),
    ("masked", 40, 40, 1040, 1536, 30, "tiled 64", True),
    ("masked", 40, 40, 1040, 512, 30, "tiled 64", True),
    ("masked", 500, 66, 16, 4608, 167, "tiled 64", False),
    ("masked", 33, 66, 1040, 640, 12, "tiled 64", True),
    ("masked", 128, 5, 1552, 3712, 128, "skinny 64x64", False),
    ("masked", 44, 3, 4160, 3712, 15, "skinny 64x64", True),
    ("masked", 600, 3, 368, 2560, 600, "skinny 32x64", False),
    ("masked", 70, 5, 1552, 2048, 1, "skinny 32x64", True),
    ("masked", 128, 5, 528, 1024, 65, "skinny 32x32", False),
    ("masked", 70, 10, 1040, 384, 36, "skinny 32x32", True),
    ("masked", 600, 5, 16, 1536, 201, "skinny 16x32", False),
    ("masked", 33, 10, 48, 2560, 12, "skinny 16x32", True),
    ("masked", 100, 3, 48, 5120, 100, "skinny 16", False),
    ("masked", 128, 3, 48, 2560, 1, "skinny 16", True),
]


class _Plan(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("block_m", ctypes.c_int), ("stream", ctypes.c_bool)]


def plan(layout, M, G, N, K, expected):
    """(kernel, whether one row tile a group reads B) by the library's own rule, with the arguments that the entry points
    give it: moe::fp4_plan(groups, rows a group, at most, rows in all, ragged, N, K)."""
    f = moe.load_library()._ZN3moe8fp4_planEidiibii
    f.argtypes = [ctypes.c_int, ctypes.c_double, ctypes.c_int, ctypes.c_int, ctypes.c_bool, ctypes.c_int, ctypes.c_int]
    f.restype = _Plan
    if layout == "dense":
        p = f(1, M, M, M, False, N, K)
    elif layout == "contiguous":
        p = f(G, M / G, M, M, True, N, K)
    else:
        p = f(G, max(1, min(expected, M)), M, G * M, True, N, K)
    return KERNELS[p.kernel], p.stream
