"""The cases that check each FP4 x FP4 kernel reach it (CPU only: the cost model runs on the host)."""
import os

import pytest

import block_scaled_fp8_dispatch_amd as moe
from fp4_kernel_cases import CASES, KERNELS, plan

pytestmark = pytest.mark.skipif(not os.path.exists(moe.LIB_PATH), reason="library not built")


@pytest.mark.parametrize("case", CASES, ids=str)
def test_case_reaches_its_kernel(case):
    kernel, stream = plan(*case[:6])
    assert kernel == case[6]
    if case[0] != "dense":
        assert stream == case[7]


def test_every_kernel_has_cases_of_every_form():
    """Each kernel in every layout, and with groups whether or not one row tile a group reads B; the 64-row one with rows of
    whole blocks of four K steps and with others, the masked layout with counts read by the product itself and through lists."""
    reached = {(c[0], c[6], c[7]) for c in CASES}
    for name in KERNELS:
        assert ("dense", name, False) in reached
        for layout in ("contiguous", "masked"):
            assert {(layout, name, False), (layout, name, True)} <= reached, (layout, name)
    for layout in ("dense", "contiguous", "masked"):
        assert {c[4] % 512 == 0 for c in CASES if c[0] == layout and c[6] == "tiled 64"} == {True, False}
    assert {c[2] > 64 for c in CASES if c[0] == "masked"} == {True, False}


def test_a_launch_stays_below_two_to_the_32_threads():
    """The largest outputs that the entry points take go to kernels whose grids one launch can hold."""
    threads = {"tiled 256": (256, 256, 256), "tiled 128": (128, 256, 256), "tiled 64": (64, 256, 256), "skinny 64x64": (64, 64, 512),
               "skinny 32x64": (32, 64, 512), "skinny 32x32": (32, 32, 512), "skinny 16x32": (16, 32, 512), "skinny 16": (16, 16, 1024)}
    for K in (128, 512, 7168, 1 << 22):
        for M in (1, 16, 300, 4096, 100000, (1 << 26) - 1):
            for N in (16, 4096, 1 << 20, (1 << 31) - 16):
                if -(-M // 128) * -(-N // 256) * 256 >= 1 << 32:
                    continue                                       # refused
                for layout, G in (("dense", 1), ("contiguous", 7), ("masked", 7)):
                    kernel, _ = plan(layout, M, G, N, K, M)
                    bm, bn, t = threads[kernel]
                    rows = G * M if layout == "masked" else M
                    if -(-rows // 128 + G) * -(-N // 256) * 256 >= 1 << 32:
                        continue
                    assert -(-rows // bm) * -(-N // bn) * t < 1 << 32, (layout, M, N, K, kernel)
