"""The dense cases of each FP4 x FP4 kernel reach the form that they name (CPU only: the cost model runs on the host)."""
import os

import pytest

import block_scaled_fp8_dispatch_amd as moe
from fp4_dense_cases import CASES
from fp4_kernel_cases import KERNELS, plan

pytestmark = pytest.mark.skipif(not os.path.exists(moe.LIB_PATH), reason="library not built")


@pytest.mark.parametrize("case", CASES, ids=str)
def test_case_reaches_its_form(case):
    M, N, K, kernel, past = case
    assert plan("dense", M, 1, N, K, 0) == (kernel, past)


def test_every_kernel_has_both_forms():
    assert {c[3:] for c in CASES} == {(k, p) for k in KERNELS for p in (False, True)}
