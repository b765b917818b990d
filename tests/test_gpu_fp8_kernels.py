"""GPU parity of every kernel of the FP8 x FP8 GEMMs on products that the cost model sends to it (fp8_kernel_cases.py), every
element against a 64-bit product. Scale bytes are random in every block and differ from row to row, so that a row or
column with another's scale shows. Tolerances as in test_gpu_fp8_gemm.py, computed on the GPU."""
import numpy as np
import pytest
import torch

from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

import block_scaled_fp8_dispatch_amd as moe  # noqa: E402
from fp8_kernel_cases import CASES, plan  # noqa: E402
from test_gpu_fp8_gemm import POISON, Problem  # noqa: E402


def values(codes, sf):
    """Codes [R, K] times a scale byte per row (or per row's 128-block) and 128 columns, in 64 bits."""
    K = codes.shape[1]
    scale = torch.exp2(sf[:, : K // 128].double() - 127)
    return (codes.view(torch.float8_e4m3fn).double().view(len(codes), K // 128, 128) * scale[:, :, None]).view(len(codes), K)


def check(p, d, rows, g):
    if len(rows) == 0:
        return
    rows = torch.as_tensor(np.asarray(rows), device="cuda")
    a, a_sf, b, b_sf = p.dev
    K = p.K
    A = values(a[rows], a_sf[rows])
    B = values(b[g], b_sf[g].repeat_interleave(128, dim=0)[: p.N])
    exact = A @ B.t()
    u = 2.0 ** -24
    gamma = (K - 1) * u / (1 - (K - 1) * u)
    bound = gamma * (A.abs() @ B.abs().t())
    if p.d_type == moe.MOE_F32:
        got = d.view(torch.float32)[rows].double()
        bound = bound + u * (exact.abs() + bound) + 2.0 ** -149
    else:
        got = d.view(torch.bfloat16)[rows].double()
        bound = bound + 2.0 ** -10 * (A.abs().view(-1, K // 8, 8).amax(2) @ B.abs().view(-1, K // 8, 8).amax(2).t())
        bound = bound + 2.0 ** -8 * (exact.abs() + bound) + 2.0 ** -134
    bad = ~((got - exact).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {torch.nonzero(bad)[0].tolist()} of group {g}"


@pytest.mark.parametrize("case", CASES, ids=str)
def test_kernel(case):
    layout, M, G, N, K, f32, expected, kernel, _ = case
    print(f"[fp8] {case}", flush=True)
    assert plan(*case[:7])[0] == kernel
    rows = G * M if layout == "masked" else M
    p = Problem(rows, N, K, G, moe.MOE_F32 if f32 else moe.MOE_BF16, seed=M + N)
    rng = np.random.default_rng(K + N)
    if layout == "dense":
        out = p.dense()
        groups = [np.arange(M)]
    elif layout == "contiguous":
        grp = rng.integers(-1, G, size=M).astype(np.int32)
        out = p.contiguous(grp)
        groups = [np.nonzero(grp == g)[0] for g in range(G)]
    else:
        cnt = rng.integers(0, M + 1, size=G).astype(np.int32)
        cnt[0], cnt[1], cnt[2] = M, 0, (M + 1) // 2
        out = p.masked(cnt, M, expected)
        groups = [g * M + np.arange(cnt[g]) for g in range(G)]
    d = torch.from_numpy(out.view(np.int32 if f32 else np.int16).copy()).cuda()
    for g, r in enumerate(groups):
        check(p, d, r, g)
    left = np.setdiff1d(np.arange(rows), np.concatenate(groups))
    assert (out[left] == POISON[p.d_type]).all(), "a row of no group was written"
