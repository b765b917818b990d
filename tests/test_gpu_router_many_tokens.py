"""The router with more than 16 experts a token and as many tokens as 2^32 threads would take at one wave each."""
import numpy as np
import pytest
import torch

from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

import block_scaled_fp8_dispatch_amd as moe  # noqa: E402
import oracle  # noqa: E402


def call(x, k):
    idx = torch.full((len(x), k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((len(x), k), -7.0, device="cuda")
    moe.moe_topk_router(idx, w, x, moe.MOE_BF16, len(x), x.shape[1], k, moe.MOE_ROUTER_SOFTMAX_CHOSEN)
    torch.cuda.synchronize()
    return idx, w


@pytest.mark.parametrize("T", [2 ** 26 - 4, 2 ** 26 + 70])
def test_a_wave_a_token(T):
    """Every token is routed, the first, middle and last ones as a call on them alone routes them."""
    print(f"[router] {T} tokens", flush=True)
    E, k = 18, 17
    x = torch.randn(T, E, dtype=torch.bfloat16, device="cuda")
    idx, w = call(x, k)
    assert int(idx.min()) >= 0 and int(idx.max()) < E and float(w.min()) > 0
    for a in (0, T // 2 - 5, 2 ** 25 - 500, 2 ** 26 - 1000, T - 1000):
        part = x[a:a + 1000].clone()
        i2, w2 = call(part, k)
        n = len(part)
        assert torch.equal(idx[a:a + n], i2) and torch.equal(w[a:a + n], w2)
        ref, _ = oracle.topk_router(part[:50].double().cpu().numpy(), k, False)
        assert np.array_equal(i2[:50].cpu().numpy(), ref)
    del x, idx, w
    torch.cuda.empty_cache()


@pytest.mark.parametrize("E,k", [(40, 17), (100, 64), (200, 20), (400, 33), (1000, 64)])
def test_several_tokens_a_wave(E, k):
    """More tokens than one pass takes, against a call on each part."""
    T, part = 140003, 30000
    x = torch.randn(T, E, device="cuda").to(torch.bfloat16)
    idx, w = call(x, k)
    for a in range(0, T, part):
        i2, w2 = call(x[a:a + part].clone(), k)
        assert torch.equal(idx[a:a + part], i2) and torch.equal(w[a:a + part], w2)
