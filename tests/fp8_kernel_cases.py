"""Products that the FP8 x FP8 GEMMs' cost model sends to each of their kernels, and a view of what it picks.

A case: layout, M (dense, contiguous: rows; masked: capacity of a group), groups, N, K, FP32 out, expected rows a
group (masked), the kernel, and whether one row tile a group reads B."""
import ctypes

import block_scaled_fp8_dispatch_amd as moe

KERNELS = ("tiled 256", "tiled 256x224", "tiled 128", "tiled 64", "skinny 64", "skinny 32", "skinny 16x32", "skinny 16")

CASES = [
    # bf16: the tiled kernels, wide stores (N % 8 == 0) and others
    ("dense", 2600, 1, 2600, 640, False, 0, "tiled 256", False),
    ("dense", 3100, 1, 4161, 1152, False, 0, "tiled 256", False),
    ("contiguous", 3100, 3, 2600, 640, False, 0, "tiled 256", False),
    ("contiguous", 2100, 10, 4161, 640, False, 0, "tiled 256", True),
    ("masked", 700, 4, 520, 256, False, 600, "tiled 256", False),
    ("masked", 70, 5, 3176, 128, False, 30, "tiled 256", True),
    ("dense", 2100, 1, 4161, 3200, False, 0, "tiled 256x224", False),
    ("dense", 3100, 1, 2600, 3200, False, 0, "tiled 256x224", False),
    ("contiguous", 1747, 10, 4161, 3200, False, 0, "tiled 256x224", True),
    ("contiguous", 3100, 3, 2600, 3200, False, 0, "tiled 256x224", False),
    ("masked", 700, 4, 3176, 3712, False, 600, "tiled 256x224", False),
    ("masked", 700, 4, 4279, 3712, False, 600, "tiled 256x224", False),
    ("contiguous", 1747, 10, 2600, 128, False, 0, "tiled 128", False),
    ("contiguous", 2600, 10, 2049, 128, False, 0, "tiled 128", False),
    ("contiguous", 1000, 10, 4161, 384, False, 0, "tiled 128", True),
    ("masked", 700, 4, 2600, 256, False, 600, "tiled 128", False),
    ("masked", 44, 27, 3176, 256, False, 22, "tiled 128", True),
    ("masked", 128, 29, 1553, 256, False, 64, "tiled 128", True),
    ("dense", 1300, 1, 2600, 384, False, 0, "tiled 64", False),
    ("contiguous", 1000, 10, 2049, 128, False, 0, "tiled 64", False),
    ("contiguous", 1000, 3, 2600, 128, False, 0, "tiled 64", False),
    ("contiguous", 16, 10, 4161, 128, False, 0, "tiled 64", True),
    ("contiguous", 600, 10, 2600, 128, False, 0, "tiled 64", True),
    ("masked", 300, 5, 2600, 128, False, 200, "tiled 64", False),
    ("masked", 1, 14, 4279, 256, False, 1, "tiled 64", True),
    ("masked", 128, 29, 520, 128, False, 64, "tiled 64", True),
    # bf16: the kernels whose waves share K
    ("dense", 1000, 1, 900, 2048, False, 0, "skinny 64", False),
    ("dense", 2100, 1, 520, 2048, False, 0, "skinny 64", False),
    ("contiguous", 1300, 3, 900, 2048, False, 0, "skinny 64", False),
    ("masked", 700, 4, 520, 3712, False, 600, "skinny 64", False),
    ("masked", 500, 3, 1553, 3712, False, 300, "skinny 64", False),
    ("dense", 600, 1, 257, 128, False, 0, "skinny 32", False),
    ("contiguous", 300, 3, 257, 128, False, 0, "skinny 32", False),
    ("masked", 300, 5, 520, 128, False, 200, "skinny 32", False),
    ("dense", 33, 1, 2600, 384, False, 0, "skinny 16x32", True),
    ("contiguous", 1000, 3, 100, 1152, False, 0, "skinny 16x32", False),
    ("masked", 70, 5, 257, 1152, False, 30, "skinny 16x32", True),
    ("dense", 100, 1, 257, 128, False, 0, "skinny 16", False),
    ("contiguous", 300, 3, 100, 384, False, 0, "skinny 16", False),
    ("masked", 500, 3, 100, 3712, False, 300, "skinny 16", False),
    # FP32
    ("dense", 2100, 1, 2049, 640, True, 0, "tiled 128", False),
    ("dense", 2100, 1, 900, 128, True, 0, "tiled 128", False),
    ("contiguous", 2600, 10, 4161, 640, True, 0, "tiled 128", False),
    ("contiguous", 300, 10, 4161, 128, True, 0, "tiled 128", True),
    ("masked", 700, 4, 900, 128, True, 600, "tiled 128", False),
    ("masked", 44, 27, 2600, 128, True, 22, "tiled 128", True),
    ("dense", 1000, 1, 2049, 384, True, 0, "skinny 64", False),
    ("dense", 2100, 1, 520, 2048, True, 0, "skinny 64", False),
    ("contiguous", 1300, 3, 1553, 384, True, 0, "skinny 64", False),
    ("contiguous", 600, 10, 4161, 2048, True, 0, "skinny 64", True),
    ("masked", 700, 4, 900, 640, True, 600, "skinny 64", False),
    ("masked", 128, 29, 2049, 1152, True, 64, "skinny 64", True),
    ("dense", 600, 1, 1553, 128, True, 0, "skinny 32", False),
    ("contiguous", 300, 3, 900, 128, True, 0, "skinny 32", False),
    ("masked", 700, 4, 257, 128, True, 600, "skinny 32", False),
    ("dense", 100, 1, 520, 128, True, 0, "skinny 16x32", False),
    ("contiguous", 600, 3, 100, 128, True, 0, "skinny 16x32", False),
    ("masked", 300, 5, 100, 128, True, 200, "skinny 16x32", False),
    ("dense", 100, 1, 257, 128, True, 0, "skinny 16", False),
    ("contiguous", 300, 3, 100, 1152, True, 0, "skinny 16", False),
    ("masked", 70, 5, 100, 256, True, 30, "skinny 16", True),
]


class _Plan(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("block_m", ctypes.c_int), ("stream", ctypes.c_bool)]


def plan(layout, M, G, N, K, f32, expected):
    """(kernel, whether one row tile a group reads B) by the library's own rule, with the arguments that the entry
    points give it: moe::fp8_plan(groups, rows a group, rows in all, ragged, N, K, FP32 out)."""
    f = moe.load_library()._ZN3moe8fp8_planEidibiib
    f.argtypes = [ctypes.c_int, ctypes.c_double, ctypes.c_int, ctypes.c_bool, ctypes.c_int, ctypes.c_int, ctypes.c_bool]
    f.restype = _Plan
    if layout == "dense":
        p = f(1, M, M, False, N, K, f32)
    elif layout == "contiguous":
        p = f(G, M / G, M, True, N, K, f32)
    else:
        p = f(G, max(1, min(expected, M)), G * M, True, N, K, f32)
    return KERNELS[p.kernel], p.stream
