"""Masked GEMMs (FP8 x FP4 and FP8 x FP8) whose capacity takes the layout launch more than one pass: every row
counted is computed, every other one left alone.

The codes stand for -2, -1, 0, 1, 2 with scales of 1, so that every sum is a whole number below 2^24: exact whatever the
order, and a bf16 output is that number rounded once."""
import pytest
import torch

from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

import block_scaled_fp8_dispatch_amd as moe  # noqa: E402

E4M3 = [0xC0, 0xB8, 0x00, 0x38, 0x40]       # -2 .. 2
E2M1 = [0xC, 0xA, 0x0, 0x2, 0x4]
K = 128


def draw(g, codes, *shape):
    at = torch.randint(0, 5, shape, generator=g, device="cuda")
    return torch.tensor(codes, dtype=torch.uint8, device="cuda")[at], at.float() - 2.0


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("G,max_m,counts", [
    (40, 20000, "some"),       # up to 800 000 rows, about half of them counted
    (3, 300000, "all"),
    (1024, 1500, "few"),       # a large capacity, hardly used
    (7, 200001, "few"),
])
def test_large_capacity(G, max_m, counts, fp4):
    print(f"[masked] {G} groups of {max_m}, {counts} fp4={fp4}", flush=True)
    N, rows = 32, G * max_m
    g = torch.Generator(device="cuda").manual_seed(G)
    a, av = draw(g, E4M3, rows, K)
    b, bv = draw(g, E2M1 if fp4 else E4M3, G, N, K)
    lo, hi = {"some": (0, max_m), "all": (max_m, max_m), "few": (0, 3)}[counts]
    cnt = torch.randint(lo, hi + 1, (G,), generator=g, device="cuda").to(torch.int32)
    a_sf = torch.full((rows, 4), 127, dtype=torch.uint8, device="cuda")
    d = torch.full((rows, N), 0x7FBF, dtype=torch.int16, device="cuda")
    if fp4:
        b = (b[..., 0::2] | (b[..., 1::2] << 4)).contiguous()
        sf = torch.full((G, N, K // 32), 127, dtype=torch.uint8, device="cuda")
        packed = torch.empty(moe.moe_gemm_packed_b_bytes(G, N, K), dtype=torch.uint8, device="cuda")
        moe.moe_gemm_prepare_b(G, N, K, b, sf, packed)
        ws = torch.full((moe.moe_gemm_workspace_bytes(rows, G),), 0xFF, dtype=torch.uint8, device="cuda")
        moe.moe_m_grouped_fp8_fp4_gemm_masked(d, a, a_sf, cnt, G, max_m, 8, N, K, packed, ws)
    else:
        sf = torch.full((G, 1, 4), 127, dtype=torch.uint8, device="cuda")
        ws = torch.full((moe.moe_fp8_gemm_workspace_bytes(rows, G),), 0xFF, dtype=torch.uint8, device="cuda")
        moe.moe_m_grouped_fp8_gemm_masked(d, moe.MOE_BF16, a, a_sf, cnt, G, max_m, 8, N, K, b, sf, ws)
    torch.cuda.synchronize()
    for i in range(G):
        n = int(cnt[i])
        at = i * max_m
        want = (av[at:at + n] @ bv[i].t().contiguous()).to(torch.bfloat16)
        assert torch.equal(d[at:at + n].view(torch.bfloat16), want), i
        assert (d[at + n:at + max_m] == 0x7FBF).all(), f"group {i}: a row past the count was written"
    del a, av, d
    torch.cuda.empty_cache()
