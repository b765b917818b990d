"""GPU parity of the FP4 x FP4 GEMMs at the longest sums that they take, bit for bit.

Codes are -1, 0 and 1 and each block's scale is 1 or 2, on both sides: products are whole numbers of at most 4, so that up to 2^22 of
them stay within 2^24 in any order of additions, FP32 holds every partial sum, and the output is the exact sum. A part of K that
is left out or counted twice, or a scale of another block, row or column, changes it. The expected sums are FP32 products of parts of
2^16 of K, exact for the same reason, added in 64 bits."""
import pytest
import torch

from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

import block_scaled_fp8_dispatch_amd as moe  # noqa: E402
from fp4_kernel_cases import plan  # noqa: E402
from test_gpu_fp4_gemm import POISON, pack  # noqa: E402

PART = 1 << 16
LONG, ODD = 1 << 22, (1 << 22) - 128


def codes(rows, K, g):
    """Packed codes [rows, K / 2] of 0, 1 and -1, and scale bytes 127 or 128 [rows, K / 32]."""
    q = torch.empty(rows, K // 2, dtype=torch.uint8, device="cuda")
    both = torch.tensor([a | b << 4 for a in (0, 2, 10) for b in (0, 2, 10)], dtype=torch.uint8, device="cuda")
    for r in range(rows):
        q[r] = both[torch.randint(0, 9, (K // 2,), generator=g, device="cuda")]
    return q, torch.randint(127, 129, (rows, K // 32), generator=g, device="cuda", dtype=torch.uint8)


def values(q, sf):
    table = torch.zeros(16, device="cuda")
    table[2], table[10] = 1.0, -1.0
    x = torch.stack((table[(q & 15).long()], table[(q >> 4).long()]), dim=2).view(len(q), -1, 32)
    return (x * (sf.float() - 126)[:, :, None]).view(len(q), -1)


def exact(a, a_sf, b, b_sf, K):
    d = torch.zeros(len(a), len(b), dtype=torch.float64, device="cuda")
    for k in range(0, K, PART):
        n = min(PART, K - k)
        A = values(a[:, k // 2:(k + n) // 2], a_sf[:, k // 32:(k + n) // 32])
        for c in range(0, len(b), 1024):
            B = values(b[c:c + 1024, k // 2:(k + n) // 2], b_sf[c:c + 1024, k // 32:(k + n) // 32])
            d[:, c:c + 1024] += (A @ B.t()).double()
    return d


CASES = [
    ("dense", 1, 1, 16, LONG, 0, "skinny 16"),
    ("dense", 3, 1, 16, ODD, 0, "skinny 16"),
    ("dense", 1000, 1, 16, LONG, 0, "skinny 16x32"),
    ("dense", 1000, 1, 16, ODD, 0, "skinny 16x32"),
    ("dense", 600, 1, 144, LONG, 0, "skinny 32x32"),
    ("dense", 1000, 1, 144, ODD, 0, "skinny 32x64"),
    ("dense", 100, 1, 4112, LONG, 0, "skinny 64x64"),
    ("dense", 100, 1, 4112, ODD, 0, "skinny 64x64"),
    ("dense", 1000, 1, 1552, LONG, 0, "tiled 64"),
    ("dense", 1000, 1, 2064, ODD, 0, "tiled 64"),
    ("dense", 1000, 1, 4112, LONG, 0, "tiled 256"),
    ("dense", 1000, 1, 4112, ODD, 0, "tiled 256"),
    ("contiguous", 1000, 3, 144, ODD, 0, "skinny 32x64"),
    ("masked", 257, 3, 2064, LONG, 257, "tiled 64"),
    ("masked", 600, 3, 4112, 1 << 20, 600, "tiled 128"),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_exact_long_sums(case):
    layout, M, G, N, K, expected, kernel = case
    print(f"[fp4] {case}", flush=True)
    assert plan(*case[:6])[0] == kernel
    g = torch.Generator(device="cuda").manual_seed(M + N)
    rows = G * M if layout == "masked" else M
    a, a_sf = codes(rows, K, g)
    b, b_sf = codes(G * N, K, g)
    packed = pack(b, b_sf, N, K, G)
    ws = torch.empty(moe.moe_fp4_gemm_workspace_bytes(rows, G), dtype=torch.uint8, device="cuda")
    d = torch.full((rows, N), POISON[moe.MOE_F32], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    if layout == "dense":
        moe.moe_fp4_gemm(d, moe.MOE_F32, a, a_sf, M, N, K, packed, ws)
        groups = [torch.arange(M, device="cuda")]
    elif layout == "contiguous":
        ids = torch.randint(-1, G, (M,), generator=g, device="cuda", dtype=torch.int32)
        moe.moe_m_grouped_fp4_gemm_contiguous(d, moe.MOE_F32, a, a_sf, ids, M, G, N, K, packed, ws)
        groups = [torch.nonzero(ids == i)[:, 0] for i in range(G)]
    else:
        count = torch.tensor([M, 0, M // 2 + 1], dtype=torch.int32, device="cuda")
        moe.moe_m_grouped_fp4_gemm_masked(d, moe.MOE_F32, a, a_sf, count, G, M, expected, N, K, packed, ws)
        groups = [i * M + torch.arange(int(count[i]), device="cuda") for i in range(G)]
    torch.cuda.synchronize()
    for i, r in enumerate(groups):
        if len(r) == 0:
            continue
        want = exact(a[r], a_sf[r], b[i * N:(i + 1) * N], b_sf[i * N:(i + 1) * N], K)
        bad = d[r].view(torch.float32).double() != want
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, first at {torch.nonzero(bad)[0].tolist()} of group {i}"
    left = torch.ones(rows, dtype=torch.bool, device="cuda")
    left[torch.cat(groups)] = False
    assert (d[left] == POISON[moe.MOE_F32]).all(), "a row of no group was written"
    del a, b, packed, d
    torch.cuda.empty_cache()
