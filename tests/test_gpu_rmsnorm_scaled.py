"""GPU parity of the norm with FP8 output on rows whose squares FP32 cannot hold, against the oracle in 64 bits; tolerances as
in test_gpu_rmsnorm.py."""
import pytest
import torch

from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

from test_gpu_rmsnorm import bf16, call, check  # noqa: E402


@pytest.mark.parametrize("cols", [256, 7168, 18432, 33024])
@pytest.mark.parametrize("large,small", [(64, -64), (64, -60), (66, -58), (80, -44), (100, -24), (126, 2), (64, 30)])
def test_small_columns_beside_a_large_one(cols, large, small):
    """One column of 2^large, which makes the row's squares infinite; the others of 2^(small - 1) to 3 * 2^small, which the root
    mean square divides into normal numbers of FP32. Each row's large column at another place; weights of about 1 and 2^20."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.rand(6, cols, generator=g, device="cuda") * 2.5 + 0.5
    x[1::2] *= -1
    x[0] = 1.3046875
    x = bf16(torch.ldexp(x, torch.tensor(small, device="cuda")))
    for r, c in enumerate((3, 0, cols - 1, 128, cols // 2, 77)):
        x[r, c] = (-1.5) ** (r & 1) * 2.0 ** large
    w = bf16(1 + 0.1 * torch.randn(cols, generator=g, device="cuda"))
    check(call(x, None, w, 1e-6), x, None, w, 1e-6)
    w = 2.0 ** 20 * w.float()
    check(call(x, None, w, 1e-6), x, None, w, 1e-6)


@pytest.mark.parametrize("cols", [256, 7168, 33024])
@pytest.mark.parametrize("top", [-126, -100, -64])
def test_rows_of_the_smallest_numbers(cols, top):
    """Rows that are scaled up: magnitudes from 2^top down to bf16's subnormal numbers, with the least eps."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(5, cols, generator=g, device="cuda").clamp(-3, 3)
    down = torch.randint(top - 7, top + 1, (5, cols), generator=g, device="cuda")
    x = bf16(torch.ldexp(x, down))
    w = 1 + 0.1 * torch.randn(cols, generator=g, device="cuda")
    check(call(x, None, w, 2.0 ** -149), x, None, w, 2.0 ** -149)


@pytest.mark.parametrize("cols", [128, 7168, 33024])
@pytest.mark.parametrize("eps", [2.0 ** 99, 2.0 ** 101, 2.0 ** 127, (2 - 2.0 ** -23) * 2.0 ** 127])
def test_large_eps(cols, eps):
    """Up to the largest finite number: rows far below, about and far above its root, and rows whose mean square and eps are
    finite each but not together."""
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.rand(7, cols, generator=g, device="cuda") + 0.5
    x[1::2] *= -1
    power = torch.tensor([-30, 0, 30, 50, 59, 64, 100], device="cuda")
    x = bf16(torch.ldexp(x, power[:, None]))
    x[4] = 1.8203125 * 2.0 ** 59
    w = bf16(1 + 0.1 * torch.randn(cols, generator=g, device="cuda"))
    check(call(x, None, w, eps), x, None, w, eps)
