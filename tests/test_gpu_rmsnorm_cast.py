"""The norm's FP8 output beside the library's own cast, `moe_cast_to_fp8`, where n is a bf16 number: byte for byte the same codes and
scales. Every h is +1 or -1 and eps far below half a step, so that the mean square's root is exactly 1 (a sum of ones, which FP32
holds) and n the weight or its negative, whatever bf16 number that is."""
import pytest
import torch

from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

import block_scaled_fp8_dispatch_amd as moe  # noqa: E402


def weights(cols, g):
    """bf16 numbers of every mantissa: each block's exponents reach from one of its own, from the smallest to the largest, down by
    up to 19; blocks of zeros and of subnormal numbers among them."""
    top = torch.randint(1, 255, (cols // 128, 1), generator=g, device="cuda")
    e = (top - torch.randint(0, 20, (cols // 128, 128), generator=g, device="cuda")).clamp(min=0)
    bits = e << 7 | torch.randint(0, 128, e.shape, generator=g, device="cuda") | torch.randint(0, 2, e.shape, generator=g, device="cuda") << 15
    if len(bits) > 4:
        bits[1] = 0
        bits[2] &= 0x807F
        bits[3] = bits[3] & 0x807F | 254 << 7
    return torch.where(bits >= 1 << 15, bits - (1 << 16), bits).to(torch.int16).view(torch.bfloat16).view(-1)


@pytest.mark.parametrize("wf32", [False, True])
@pytest.mark.parametrize("rows,cols", [(3, 128), (5, 640), (16, 7168), (600, 7168), (1100, 4096), (700, 10240), (520, 16384), (9, 18432), (3, 33024)])
def test_same_bytes_as_the_cast(rows, cols, wf32):
    print(f"[norm] {rows} x {cols} {wf32}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(cols)
    w = weights(cols, g)
    x = (1 - 2 * torch.randint(0, 2, (rows, cols), generator=g, device="cuda")).to(torch.bfloat16)
    stride = 4 * -(-cols // 512)
    q, cast_q = (torch.full((rows, cols), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(2))
    sf, cast_sf = (torch.full((rows, stride), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(2))
    normed = torch.empty_like(x)
    moe.moe_rmsnorm_to_fp8(q, sf, normed, None, x, None, w.float() if wf32 else w, moe.MOE_F32 if wf32 else moe.MOE_BF16, rows, cols, 2.0 ** -60)
    torch.cuda.synchronize()
    n = torch.where(x > 0, w.view(torch.int16), w.view(torch.int16) ^ -2 ** 15)
    assert torch.equal(normed.view(torch.int16), n), "normed"
    moe.moe_cast_to_fp8(normed, rows, cols, cast_q, cast_sf)
    torch.cuda.synchronize()
    assert torch.equal(sf, cast_sf), "scale bytes"
    assert torch.equal(q, cast_q), "codes"
    assert cols < 1024 or len(torch.unique(sf)) > 4 and len(torch.unique(q)) > 100
