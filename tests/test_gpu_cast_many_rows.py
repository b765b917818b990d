"""The cast of more rows than one launch of fewer than 2^32 threads takes."""
import pytest
import torch

from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

import block_scaled_fp8_dispatch_amd as moe  # noqa: E402


def test_cast_of_many_rows():
    """2^26 + 4099 rows: each row as a cast of its part alone gives it."""
    rows, cols = 2 ** 26 + 4099, 128
    print(f"[cast] {rows} x {cols}", flush=True)
    x = torch.randn(rows, cols, dtype=torch.bfloat16, device="cuda")
    q = torch.full((rows, cols), 0x5A, dtype=torch.uint8, device="cuda")
    sf = torch.full((rows, 4), 0x5A, dtype=torch.uint8, device="cuda")
    moe.moe_cast_to_fp8(x, rows, cols, q, sf)
    torch.cuda.synchronize()
    part = 2 ** 24
    for a in range(0, rows, part):
        n = min(part, rows - a)
        q2, sf2 = torch.empty(n, cols, dtype=torch.uint8, device="cuda"), torch.empty(n, 4, dtype=torch.uint8, device="cuda")
        moe.moe_cast_to_fp8(x[a:a + n], n, cols, q2, sf2)
        torch.cuda.synchronize()
        assert torch.equal(q[a:a + n], q2) and torch.equal(sf[a:a + n], sf2), a
        del q2, sf2
    del x, q, sf
    torch.cuda.empty_cache()
