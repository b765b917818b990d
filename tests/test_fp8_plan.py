"""The cases that check each FP8 x FP8 kernel reach it (CPU only: the cost model runs on the host)."""
import os

import pytest

import block_scaled_fp8_dispatch_amd as moe
from fp8_kernel_cases import CASES, KERNELS, plan

pytestmark = pytest.mark.skipif(not os.path.exists(moe.LIB_PATH), reason="library not built")


@pytest.mark.parametrize("case", CASES, ids=str)
def test_case_reaches_its_kernel(case):
    kernel, stream = plan(*case[:7])
    assert kernel == case[7]
    if case[0] != "dense":
        assert stream == case[8]


def test_every_kernel_has_cases_of_every_form():
    """Each kernel of each output type in every layout; the tiled ones with rows that allow wide stores and with others;
    the 64-row one both where one row tile a group reads B and where several do."""
    reached = {(c[0], c[5], c[7]) for c in CASES}
    for f32 in (False, True):
        for name in KERNELS:
            if f32 and name.startswith("tiled") and name != "tiled 128":
                continue
            for layout in ("dense", "contiguous", "masked"):
                # dense bf16 products of many rows go to 256-row tiles rather than 128
                if (layout, f32, name) == ("dense", False, "tiled 128"):
                    continue
                assert (layout, f32, name) in reached, (layout, f32, name)
    for name in ("tiled 256", "tiled 128", "tiled 64"):
        assert {c[3] % 8 == 0 for c in CASES if c[7] == name and not c[5]} == {True, False}
    assert {(c[3] % 8 == 0, c[8]) for c in CASES if c[7] == "tiled 64" and c[0] != "dense"} == {
        (True, True), (True, False), (False, True), (False, False)}
