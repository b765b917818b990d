"""GPU tests of the norm with FP8 output on rows of so many columns that a thread takes them in turn.

`test_powers_of_two`: h is +1 or -1 and the weights are powers of two, so that the mean of the squares is 1 but for the sums'
rounding and eps, n is +-2^k but for less than a thousandth, and every output byte is known. Signs, weights and the largest
weight of a block follow a hash of the column, so that a column with another's shows."""
import pytest
import torch

from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

import block_scaled_fp8_dispatch_amd as moe  # noqa: E402

GUARD = 4096
PART = 1 << 26


def mix(c):
    c = (c * 0x9E3779B1 + 0x7F4A7C15) & 0xFFFFFFFF
    c = ((c ^ (c >> 15)) * 0x85EBCA6B) & 0xFFFFFFFF
    return c ^ (c >> 13)


def parts(cols):
    for at in range(0, cols, PART):
        yield at, min(PART, cols - at)


def columns(row, at, n):
    """(sign of h, exponent of the weight, exponent of the block's largest weight) of columns at .. at+n-1."""
    c = torch.arange(at, at + n, device="cuda")
    top = (mix(c >> 7) & 7) - 3
    e = top - (mix(c + 7) >> 5 & 7)
    e = torch.where(c & 127 == mix(c >> 7) >> 8 & 127, top, e)       # a column of every block has the largest
    return 1 - 2 * (mix(c + row * 40503) >> 3 & 1), e, top


@pytest.mark.parametrize("rows,cols", [(2, 33024), (3, 2 ** 20 + 128), (1, 2 ** 31 - 8192), (1, 2 ** 31 - 128)])
def test_powers_of_two(rows, cols):
    """Up to the most columns that the entry point takes."""
    print(f"[norm] {rows} x {cols}", flush=True)
    stride = 4 * -(-cols // 512)
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    w = torch.empty(cols, dtype=torch.bfloat16, device="cuda")
    for at, n in parts(cols):
        for r in range(rows):
            sign, e, _ = columns(r, at, n)
            x[r, at:at + n] = sign
        w[at:at + n] = torch.exp2(e.float())
    q = torch.full((rows * cols + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
    sf = torch.full((rows * stride + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
    normed = torch.full((rows * cols + GUARD,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = torch.full((rows * cols + GUARD,), 7.0, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    moe.moe_rmsnorm_to_fp8(q, sf, normed, out, x, None, w, moe.MOE_BF16, rows, cols, 1e-12)
    torch.cuda.synchronize()
    for t, guard in ((q, 0xA5), (normed, 7.0), (out, 7.0)):
        assert (t[rows * cols:] == guard).all(), "a store went past the end"
    assert (sf[rows * stride:] == 0xA5).all(), "a store went past the end"
    for r in range(rows):
        for at, n in parts(cols):
            sign, e, top = columns(r, at, n)
            i = r * cols + at
            assert torch.equal(out[i:i + n], x[r, at:at + n]), (r, at)
            assert torch.equal(normed[i:i + n].float(), sign * torch.exp2(e.float())), (r, at)
            # 2^top is 1.75 * 2^8 or less from 2^(top - 8) on: codes of 2^(e - top + 8), exponents of 7 more
            assert torch.equal(q[i:i + n].long(), (e - top + 8 + 7) * 8 + (1 - sign) * 64), (r, at)
            b = r * stride + (at >> 7)
            assert torch.equal(sf[b:b + n // 128].long(), top[::128] - 8 + 127), (r, at)
        assert not sf[r * stride + cols // 128:(r + 1) * stride].any(), "scale bytes past the row's last block"
    del x, w, q, sf, normed, out
    torch.cuda.empty_cache()
