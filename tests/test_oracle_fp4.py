"""Pins of the 4-bit oracle and of the norm's (CPU): closed forms, the generator's own quantiser, torch in float64."""
import numpy as np
import torch

import oracle
from synth.generate import cast_fp4_blocks


def test_e2m1_codes():
    mags = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert oracle.encode_e2m1_rne(np.array(mags)).tolist() == list(range(8))
    assert oracle.encode_e2m1_rne(-np.array(mags, dtype=float)).tolist() == [c | 8 for c in range(8)]
    # midpoints go to the even code, and what is next to one to its side
    mid = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    assert oracle.encode_e2m1_rne(mid).tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert oracle.encode_e2m1_rne(mid + 1e-9).tolist() == [1, 2, 3, 4, 5, 6, 7]
    assert oracle.encode_e2m1_rne(mid - 1e-9).tolist() == [0, 1, 2, 3, 4, 5, 6]
    assert oracle.encode_e2m1_rne(np.array([-0.0, -0.1, 0.1])).tolist() == [8, 8, 0]


def test_scale_exponent():
    a = np.array([0.0, 6.0, np.nextafter(6.0, 7), 3.0, 3.0000001, 0.75, 6 * 2.0 ** -100, 6.1 * 2.0 ** -100, 2.0 ** -140, 3.4e38])
    assert oracle.fp4_exponent(a).tolist() == [0, 0, 1, -1, 0, -3, -100, -99, -127, 126]


def test_cast_hand_worked():
    x = np.zeros((1, 64))
    x[0, :5] = [6.0, -0.25, 2.5, -5.0, 0.1]
    x[0, 32:35] = [0.375, -0.0625, 1e-30]                      # s = -4: 6, -1, 0
    q, sf = oracle.cast_to_fp4(x)
    assert sf.tolist() == [[127, 123]]
    assert q[0, :3].tolist() == [0x7 | 0x8 << 4, 0x4 | 0xE << 4, 0x0] and q[0, 16:18].tolist() == [0x7 | 0xA << 4, 0]
    v = oracle.cast_from_fp4(q, sf)
    assert v[0, :5].tolist() == [6.0, 0.0, 2.0, -4.0, 0.0] and v[0, 32:35].tolist() == [0.375, -0.0625, 0.0]
    x[0, 40], x[0, 3] = np.inf, np.nan
    q, sf = oracle.cast_to_fp4(x)
    assert sf.tolist() == [[255, 255]] and not q.any() and np.isnan(oracle.cast_from_fp4(q, sf)).all()


def test_cast_against_the_generators_quantiser():
    g = torch.Generator().manual_seed(4)
    x = torch.randn(33, 160, generator=g) * torch.exp2(torch.randint(-30, 30, (33, 1), generator=g).float())
    x[3, 32:64] = 0
    x[5] = (x[5] * 8).round() / 8                               # ties
    q, sf = oracle.cast_to_fp4(x.double().numpy())
    want_q, want_sf = cast_fp4_blocks(x)
    assert np.array_equal(q, want_q.numpy()) and np.array_equal(sf, want_sf.numpy())
    # what the codes stand for casts to itself, where a block reaches the upper half of the range
    v = oracle.cast_from_fp4(q, sf)
    q2, sf2 = oracle.cast_to_fp4(v)
    assert np.array_equal(oracle.cast_from_fp4(q2, sf2), v)


def test_gemm_against_torch():
    rng = np.random.default_rng(1)
    a, b = rng.integers(0, 256, (7, 128)).astype(np.uint8), rng.integers(0, 256, (16, 128)).astype(np.uint8)
    a_sf, b_sf = rng.integers(120, 134, (7, 8)).astype(np.uint8), rng.integers(120, 134, (16, 8)).astype(np.uint8)
    A, B = torch.from_numpy(oracle.cast_from_fp4(a, a_sf)), torch.from_numpy(oracle.cast_from_fp4(b, b_sf))
    r = oracle.fp4_gemm(a, a_sf, b, b_sf, 256)
    np.testing.assert_allclose(r["exact"], (A @ B.T).numpy(), rtol=1e-13, atol=1e-13)
    assert (r["bound"] > 0).all() and (r["bound"] < 1e-3 * (A.abs() @ B.abs().T).numpy()).all()


def test_rmsnorm():
    x, w = np.array([[3.0, 4.0], [0.0, 0.0]]), np.array([1.0, -2.0])
    h, n = oracle.rmsnorm(x, None, w, 12.5)
    assert np.array_equal(h, x)
    np.testing.assert_allclose(n, [[3 / 5.0, -8 / 5.0], [0, 0]], rtol=1e-15)
    h, n = oracle.rmsnorm(x, np.array([[2.0 ** -30, 1.0], [5.0, 12.0]]), w, 1e-6)
    assert h.tolist() == [[3.0, 5.0], [5.0, 12.0]]                # the sum in FP32
    t = torch.tensor(h)
    want = torch.nn.functional.rms_norm(t, (2,), torch.tensor(w), eps=float(np.float32(1e-6)))
    np.testing.assert_allclose(n, want.numpy(), rtol=1e-13)
