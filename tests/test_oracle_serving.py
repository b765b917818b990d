"""Pins of the serving oracle (CPU): the router against hand-worked rows and torch's sort and
softmax, the FP8 block GEMM against torch's decoders."""
import math

import numpy as np
import torch

import oracle


def test_router_hand_worked():
    inf, nan = math.inf, math.nan
    x = np.array([[0.0, 1.0, 1.0, -1.0], [-inf, -inf, 2.0, nan], [-inf, nan, -inf, -inf], [-0.0, 0.0, -1.0, inf]])
    idx, w = oracle.topk_router(x, 2, False)
    assert idx.tolist() == [[1, 2], [2, -1], [-1, -1], [3, 0]]
    assert w.tolist() == [[0.5, 0.5], [1.0, 0.0], [0.0, 0.0], [1.0, 0.0]]
    idx, w = oracle.topk_router(x, 1, True, 3.0)
    e = math.exp
    assert idx[:, 0].tolist() == [1, 2, -1, 3]
    np.testing.assert_allclose(w[:, 0], [3.0 / (2 + e(-1) + e(-2)), 3.0, 0.0, 3.0], rtol=1e-14)


def test_router_against_torch():
    x = torch.randn(50, 37, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    x[:, 5] = x[:, 20]
    idx, w = oracle.topk_router(x.numpy(), 6, False)
    top, order = torch.sort(x, dim=1, descending=True, stable=True)
    assert np.array_equal(idx, order[:, :6].numpy())
    np.testing.assert_allclose(w, torch.softmax(top[:, :6], 1).numpy(), rtol=1e-12)
    _, wa = oracle.topk_router(x.numpy(), 6, True)
    np.testing.assert_allclose(wa, torch.softmax(x, 1).gather(1, order[:, :6]).numpy(), rtol=1e-12)


def test_fp8_gemm_against_torch_decoders():
    rng = np.random.default_rng(3)
    M, N, K = 5, 200, 384
    a = rng.integers(0, 256, (M, K)).astype(np.uint8)
    b = rng.integers(0, 256, (N, K)).astype(np.uint8)
    a[(a & 0x7F) == 0x7F] = 0
    b[(b & 0x7F) == 0x7F] = 1
    a_sf = rng.integers(120, 134, (M, 4)).astype(np.uint8)
    b_sf = rng.integers(120, 134, (2, 4)).astype(np.uint8)

    def dec(c):
        return torch.from_numpy(c).view(torch.float8_e4m3fn).double()
    A = dec(a) * torch.from_numpy(a_sf[:, :3]).view(torch.float8_e8m0fnu).double().repeat_interleave(128, 1)
    sb = torch.from_numpy(b_sf[:, :3].copy()).view(torch.float8_e8m0fnu).double()
    B = dec(b) * sb.repeat_interleave(128, 1).repeat_interleave(128, 0)[:N]
    r = oracle.fp8_gemm(a, a_sf, b, b_sf, K)
    np.testing.assert_allclose(r["exact"], (A @ B.T).numpy(), rtol=1e-12)
    assert (r["bound"] > 0).all()
    assert oracle.gemm_f32_within_bound(r["exact"].astype(np.float32), r["exact"], r["bound"]).all()
    assert not oracle.gemm_f32_within_bound(r["exact"] + 3 * r["bound"], r["exact"], r["bound"]).any()
