"""GPU tests of the norm with FP8 output on rows of so many columns that a thread takes them in turn.

`test_powers_of_two`: h is +1 or -1 and the weights are powers of two, so that the mean of the squares is 1 but for the sums'
rounding and eps, n is +-2^k but for less than a thousandth, and every output byte is known. Signs, weights and the largest
weight of a block follow a hash of the column, so that a column with another's shows.

`test_sum_of_many_squares`: n against 64 bits, with a bound that does not grow with the row. Each square is off by 2^-24 relative,
8 of them are added (7 roundings), chunks in 64 bits (nothing to count), their sum rounded (1), and 1024 threads' added over 16
lanes, four rows and 16 waves (4 + 2 + 4): the sum of positive numbers within 20 * 2^-24 of itself, its root within 10; the
division by the columns, their count in FP32, eps, the root, the reciprocal and the two products at most 8 more. Second orders
are far below the 2 that make it 20 * 2^-24."""
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


@pytest.mark.parametrize("value", [1.3046875, 1.0078125, -1.703125])
@pytest.mark.parametrize("cols", [2 ** 20, 2 ** 26, 2 ** 30, 2 ** 31 - 128])
def test_sum_of_many_squares(cols, value):
    """Equal columns, whose squares all round the same way when they are added to a large sum."""
    print(f"[norm] {cols} of {value}", flush=True)
    delta = 20 * 2.0 ** -24
    x = torch.full((1, cols), value, dtype=torch.bfloat16, device="cuda")
    period = torch.linspace(1, 2, 2 ** 15 + 128, dtype=torch.float32, device="cuda")
    w = period.repeat(cols // len(period) + 1)[:cols].clone()
    q = torch.empty(1, cols, dtype=torch.uint8, device="cuda")
    sf = torch.empty(1, 4 * -(-cols // 512), dtype=torch.uint8, device="cuda")
    normed = torch.empty(1, cols, dtype=torch.bfloat16, device="cuda")
    moe.moe_rmsnorm_to_fp8(q, sf, normed, None, x, None, w, moe.MOE_F32, 1, cols, 1e-6)
    torch.cuda.synchronize()
    r = value / (value * value + 1e-6) ** 0.5
    for at, n in parts(cols):
        exact = r * w[at:at + n].double()
        slack = delta * exact.abs()
        half = torch.exp2(torch.floor(torch.log2(exact.abs() + slack)) - 8)          # half a bf16 step there
        assert ((normed[0, at:at + n].double() - exact).abs() <= half + slack).all(), at
        # codes at the scale of 2^0 to 2 (1.75 * 2^8 * 2^-8 is below 2): half a step of 8 in a binade
        scale = torch.exp2(sf[0, at >> 7:(at + n) >> 7].double() - 127).repeat_interleave(128)
        got = q[0, at:at + n].view(torch.float8_e4m3fn).double() * scale
        half = torch.exp2(torch.floor(torch.log2(exact.abs() + slack)) - 4)
        assert ((got - exact).abs() <= half + slack).all(), at
    del x, w, q, sf, normed
    torch.cuda.empty_cache()
