"""GPU parity of every kernel of the FP4 x FP4 GEMMs on products that the cost model sends to it (fp4_kernel_cases.py), every
element against a 64-bit product. Scale bytes are random in every block of 32 and differ from row to row, so that a row or
column with another's scale shows. Tolerances as in test_gpu_fp4_gemm.py, computed on the GPU."""
import numpy as np
import pytest
import torch

from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

import block_scaled_fp8_dispatch_amd as moe  # noqa: E402
from fp4_kernel_cases import CASES, plan  # noqa: E402
from test_gpu_fp4_gemm import POISON, TYPES, Problem  # noqa: E402

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def values(codes, sf):
    """Rows of packed codes [R, K / 2], low halves first, with a scale byte per 32, in 64 bits."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device="cuda")
    x = torch.stack((codes & 15, codes >> 4), dim=2).long()
    x = table[x].view(len(codes), -1, 32) * torch.exp2(sf.double() - 127)[:, :, None]
    return x.view(len(codes), -1)


def check(p, d, rows, g):
    if len(rows) == 0:
        return
    rows = torch.as_tensor(np.asarray(rows), device="cuda")
    K = p.K
    A = values(p.ga[rows], p.ga_sf[rows])
    B = values(torch.from_numpy(p.b[g]).cuda(), torch.from_numpy(p.b_sf[g]).cuda())
    exact = A @ B.t()
    u = 2.0 ** -24
    bound = (K - 1) * u / (1 - (K - 1) * u) * (A.abs() @ B.abs().t())
    if p.d_type == moe.MOE_F32:
        got = d.view(torch.float32)[rows].double()
        bound = bound + u * (exact.abs() + bound) + 2.0 ** -149
    else:
        got = d.view(torch.bfloat16)[rows].double()
        bound = bound + 2.0 ** -8 * (exact.abs() + bound) + 2.0 ** -134
    bad = ~((got - exact).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {torch.nonzero(bad)[0].tolist()} of group {g}"


@pytest.mark.parametrize("d_type", TYPES)
@pytest.mark.parametrize("case", CASES, ids=str)
def test_kernel(case, d_type):
    layout, M, G, N, K, expected, kernel, _ = case
    print(f"[fp4] {case} {d_type}", flush=True)
    assert plan(*case[:6])[0] == kernel
    rows = G * M if layout == "masked" else M
    p = Problem(rows, N, K, G, d_type, seed=M + N)
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
    d = torch.from_numpy(out.view(np.int32 if d_type == moe.MOE_F32 else np.int16).copy()).cuda()
    for g, r in enumerate(groups):
        check(p, d, r, g)
    left = np.setdiff1d(np.arange(rows), np.concatenate(groups))
    assert (out[left] == POISON[d_type]).all(), "a row of no group was written"


@pytest.mark.parametrize("G", [63, 64, 65, 130])
@pytest.mark.parametrize("max_m", [1, 40, 300])
def test_counts_at_the_border_of_a_wave(G, max_m):
    """Up to 64 groups every wave sums the counts itself; more are listed by a launch before. Empty groups at both ends and in
    runs, one that fills its capacity, counts out of range."""
    N, K = 80, 256
    print(f"[fp4] {G} groups of {max_m}", flush=True)
    p = Problem(G * max_m, N, K, G, moe.MOE_F32, seed=G)
    rng = np.random.default_rng(G + max_m)
    cnt = np.where(rng.random(G) < 0.4, 0, rng.integers(0, max_m + 1, size=G)).astype(np.int32)
    cnt[0], cnt[-1], cnt[G // 2], cnt[G // 2 + 1] = 0, -3, max_m, max_m + 9
    c = np.clip(cnt, 0, max_m)
    for cnt, c in ((cnt, c), (cnt[::-1].copy(), c[::-1].copy())):
        out = p.masked(cnt, max_m, int(max(1, c.mean())))
        d = torch.from_numpy(out.view(np.int32).copy()).cuda()
        written = np.concatenate([g * max_m + np.arange(c[g]) for g in range(G)])
        for g in range(G):
            check(p, d, g * max_m + np.arange(c[g]), g)
        assert (out[np.setdiff1d(np.arange(G * max_m), written)] == POISON[moe.MOE_F32]).all(), "a row past a count was written"
