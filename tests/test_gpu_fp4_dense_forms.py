"""GPU parity of the dense FP4 x FP4 GEMM on products that reach each kernel with B read past the caches and not
(fp4_dense_cases.py), every element against a 64-bit product, as in test_gpu_fp4_kernels.py."""
import numpy as np
import pytest
import torch

from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

import block_scaled_fp8_dispatch_amd as moe  # noqa: E402
from fp4_dense_cases import CASES  # noqa: E402
from fp4_kernel_cases import plan  # noqa: E402
from test_gpu_fp4_gemm import TYPES, Problem  # noqa: E402
from test_gpu_fp4_kernels import check  # noqa: E402


@pytest.mark.parametrize("d_type", TYPES)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_form(case, d_type):
    M, N, K, kernel, past = case
    print(f"[fp4] {case} {d_type}", flush=True)
    assert plan("dense", M, 1, N, K, 0) == (kernel, past)
    p = Problem(M, N, K, 1, d_type, seed=M + N)
    out = p.dense()
    check(p, torch.from_numpy(out.view(np.int32 if d_type == moe.MOE_F32 else np.int16).copy()).cuda(), np.arange(M), 0)
