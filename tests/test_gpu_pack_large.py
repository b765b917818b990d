"""Packing of more weights than one launch of fewer than 2^32 threads takes."""
import pytest
import torch

from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

import block_scaled_fp8_dispatch_amd as moe  # noqa: E402


def test_packing_of_64_gib():
    """B of 17 groups of 4 GiB: every group packed as a call on it alone packs it."""
    G, N, K = 17, 65536, 131072
    group = N * K // 2
    print(f"[pack] {G} groups of {group} bytes", flush=True)
    b = torch.empty(G * group, dtype=torch.uint8, device="cuda")
    for i in range(G):
        b[i * group:(i + 1) * group].random_(0, 256)
    b_sf = torch.randint(0, 255, (G, N, K // 32), dtype=torch.uint8, device="cuda")
    data, scales = group, N * K // 32                     # N a multiple of 256, K of 512: no padding
    packed = torch.full((moe.moe_gemm_packed_b_bytes(G, N, K),), 0x5A, dtype=torch.uint8, device="cuda")
    assert packed.numel() == G * (data + scales)
    moe.moe_gemm_prepare_b(G, N, K, b, b_sf, packed)
    one = torch.empty(moe.moe_gemm_packed_b_bytes(1, N, K), dtype=torch.uint8, device="cuda")
    for i in range(G):
        moe.moe_gemm_prepare_b(1, N, K, b[i * group:(i + 1) * group], b_sf[i], one)
        torch.cuda.synchronize()
        assert torch.equal(packed[i * data:(i + 1) * data], one[:data]), i
        assert torch.equal(packed[G * data + i * scales:G * data + (i + 1) * scales], one[data:]), i
    del b, b_sf, packed, one
    torch.cuda.empty_cache()
