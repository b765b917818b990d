"""GPU parity of the norm with FP8 output against the oracle in 64 bits.

residual_out is the FP32 sum's bf16, bit for bit. n is FP32 arithmetic: the mean of the squares is a sum of `cols` positive
terms, each with three roundings, added in chains of at most cols / 256 + 72 numbers in any thread and across threads, so its
relative error is below (cols / 256 + 80) * 2^-24 (scaling by powers of two is exact); the square root halves it; its own
rounding, the division, the two by `cols` and eps and the three products add at most 8 * 2^-24. Together
    delta = (cols / 512 + 48) * 2^-24.
normed is n's bf16: within delta |n| and half a bf16 step (2^-8 relative of the rounded value, 2^-134 at the bottom). The scale byte is
the rule's for some largest magnitude within delta of the exact one, and each code the e4m3 number nearest to a value within
delta of n (half a step: 2^-4 relative, 2^-10 below the smallest normal number, at the block's scale)."""
import numpy as np
import pytest
import torch

from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

import block_scaled_fp8_dispatch_amd as moe  # noqa: E402
import oracle  # noqa: E402

GUARD = 512


def bf16(t):
    return t.to(torch.bfloat16)


def call(x, res, w, eps, normed=True, out=True, stream=None):
    """(codes, scale bytes, normed or None, residual_out or None) with guards behind every output."""
    R, C = x.shape
    sfw = 4 * -(-C // 512)
    q = torch.full((R * C + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
    sf = torch.full((R * sfw + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
    n = torch.full((R * C + GUARD,), 0x5A5A, dtype=torch.int16, device="cuda") if normed else None
    o = torch.full((R * C + GUARD,), 0x5A5A, dtype=torch.int16, device="cuda") if out else None
    torch.cuda.synchronize()
    moe.moe_rmsnorm_to_fp8(q, sf, n, o, x, res, w, moe.MOE_F32 if w.dtype == torch.float32 else moe.MOE_BF16, R, C, eps,
                           stream=stream)
    torch.cuda.synchronize()
    assert (q[R * C:] == 0xA5).all() and (sf[R * sfw:] == 0xA5).all(), "a store went past the end"
    for t in (n, o):
        assert t is None or (t[R * C:] == 0x5A5A).all(), "a store went past the end"
    cut = lambda t: None if t is None else t[: R * C].view(R, C).cpu().numpy().view(np.uint16)  # noqa: E731
    return q[: R * C].view(R, C).cpu().numpy(), sf[: R * sfw].view(R, sfw).cpu().numpy(), cut(n), cut(o)


def check(got, x, res, w, eps):
    q, sf, normed, out = got
    R, C = x.shape
    f64 = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    h, n = oracle.rmsnorm(f64(x), f64(res), f64(w), eps)
    delta = (C / 512 + 48) * 2.0 ** -24
    if out is not None:
        assert np.array_equal(out, oracle.bf16_rne_bits(h)), "residual_out"
    if normed is not None:
        v = oracle.bf16_bits_to_f64(normed)
        assert (np.abs(v - n) <= delta * np.abs(n) + 2.0 ** -8 * np.abs(n) * (1 + delta) + 2.0 ** -134).all(), "normed"
    nb = C // 128
    blocks = n.reshape(R, nb, 128)
    amax = np.abs(blocks).max(-1)
    lo, hi = (np.where(amax == 0, 0, np.maximum(oracle.pow2_scale_exponent(a), -127)) for a in (amax * (1 - delta), amax * (1 + delta)))
    s = sf[:, :nb].astype(np.int64) - 127
    assert ((s >= lo) & (s <= hi)).all(), "scale bytes"
    assert not sf[:, nb:].any(), "scale bytes past the row's last block"
    scale = 2.0 ** s[..., None].astype(np.float64)
    v = oracle.decode_e4m3(q).reshape(R, nb, 128) * scale
    slack = delta * np.abs(blocks) + 2.0 ** -148               # (three products may round among the subnormal numbers)
    # half a step of the binade of the larger of the two neighbours: 2^-4 of it
    step = np.maximum(2.0 ** -4 * np.maximum(np.abs(v), np.abs(blocks) + slack), 2.0 ** -10 * scale)
    assert (np.abs(v - blocks) <= step + slack).all(), "codes"
    # and nearest: no neighbouring code is nearer by more than the slack allows
    for d in (-1, 1):
        mag = (q & 0x7F).astype(np.int64) + d
        ok = (mag >= 0) & (mag <= 0x7E)
        other = oracle.decode_e4m3(((q & 0x80) | np.clip(mag, 0, 0x7E)).astype(np.uint8)).reshape(R, nb, 128) * scale
        nearer = np.abs(other - blocks) < np.abs(v - blocks) - 2 * slack
        assert not (nearer & ok.reshape(R, nb, 128)).any(), "a nearer code exists"


def rows(R, C, seed, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return bf16(torch.randn(R, C, generator=g, device="cuda") * spread)


SIZES = [(1, 128), (2, 256), (16, 384), (33, 640), (7, 1152), (5, 2048), (9, 2176), (16, 7168), (3, 8192), (4, 10368), (2, 16384),
         (3, 18432), (2, 33024), (1025, 128), (513, 512), (300, 4096)]


@pytest.mark.parametrize("wf32", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("R,C", SIZES)
def test_norm(R, C, residual, wf32):
    print(f"[norm] {R} {C} {residual} {wf32}", flush=True)
    x = rows(R, C, R + C)
    res = rows(R, C, R + C + 1, 5.0) if residual else None
    w = 1 + 0.2 * torch.randn(C, generator=torch.Generator(device="cuda").manual_seed(C), device="cuda")
    w = w if wf32 else bf16(w)
    got = call(x, res, w, 1e-6)
    check(got, x, res, w, 1e-6)
    again = call(x, res, w, 1e-6)
    assert all(np.array_equal(a, b) for a, b in zip(got, again)), "two calls gave different bytes"
    # the optional outputs change nothing
    some = call(x, res, w, 1e-6, normed=False, out=False)
    assert np.array_equal(some[0], got[0]) and np.array_equal(some[1], got[1])


@pytest.mark.parametrize("C", [128, 640, 7168, 18432])
@pytest.mark.parametrize("eps", [1e-6, 1e-30, 1e-38, 3.0])
def test_magnitudes(C, eps):
    """Rows from 2^-126 to the top of bf16, whose squares leave FP32's range both ways, a zero row, and one with a single
    number: each against the formula."""
    g = torch.Generator(device="cuda").manual_seed(C)
    x = torch.randn(13, C, generator=g, device="cuda").clamp(-3, 3)
    power = torch.tensor([-126, -110, -75, -66, -62, -40, 0, 40, 60, 66, 90, 126, 0], device="cuda")
    x = bf16(torch.ldexp(x, power[:, None]))
    x[6] = 0
    x[12] = 0
    x[12, C - 3] = -2.0 ** 100
    w = bf16(1 + 0.1 * torch.randn(C, generator=g, device="cuda"))
    check(call(x, None, w, eps), x, None, w, eps)


@pytest.mark.parametrize("C", [256, 7168, 18432])
def test_infinities_and_nan(C):
    """An infinity: its block NaN, the row's other columns 0. A NaN, or a sum that is one: the whole row. Other rows stay."""
    x, res = rows(6, C, 1), rows(6, C, 2)
    w = torch.ones(C, device="cuda")
    clean = call(x, res, w, 1e-6)
    x[1, 130] = float("inf")
    x[3, C - 1] = float("nan")
    x[4, 0], res[4, 0] = float("inf"), -float("inf")
    q, sf, normed, out = call(x, res, w, 1e-6)
    for r in (0, 2, 5):
        for a, b in zip((q, sf, normed, out), clean):
            assert np.array_equal(a[r], b[r])
    n = oracle.bf16_bits_to_f64(normed)
    nan = np.zeros((6, C), dtype=bool)
    nan[1, 130] = True
    nan[[3, 4]] = True
    assert np.isnan(n[nan]).all() and (n[1][~nan[1]] == 0).all()
    nb = C // 128
    assert (sf[1, :nb] == np.where(np.arange(nb) == 1, 255, 127)).all() and (sf[[3, 4], :nb] == 255).all()
    assert ((q[1, 128:256] & 0x7F) == 0x7F).all() and ((q[[3, 4]] & 0x7F) == 0x7F).all()
    assert (np.delete(q[1].reshape(nb, 128), 1, axis=0) & 0x7F == 0).all()


@pytest.mark.parametrize("C", [384, 7168, 18432])
def test_in_place(C):
    """residual_out may be the residual, or x."""
    x, res = rows(9, C, 3), rows(9, C, 4)
    w = bf16(torch.ones(C, device="cuda"))
    want = call(x, res, w, 1e-5)
    for which in (0, 1):
        t = [x.clone(), res.clone()]
        q = torch.empty(9, C, dtype=torch.uint8, device="cuda")
        sf = torch.empty(9, 4 * -(-C // 512), dtype=torch.uint8, device="cuda")
        moe.moe_rmsnorm_to_fp8(q, sf, None, t[which], t[0], t[1], w, moe.MOE_BF16, 9, C, 1e-5)
        torch.cuda.synchronize()
        assert np.array_equal(q.cpu().numpy(), want[0]) and np.array_equal(sf.cpu().numpy(), want[1])
        assert np.array_equal(t[which].view(torch.int16).cpu().numpy().view(np.uint16), want[3])
        assert torch.equal(t[1 - which], (x, res)[1 - which])


def test_matches_the_cast_where_n_is_a_bf16_number():
    """With a row whose root mean square is exactly 1 and unit weights n is x (eps below half a step): the FP8 cast's bytes."""
    x = torch.ones(4, 512, device="cuda")
    x[:, ::2] = -1
    x[2, :128] *= 2.0 ** -0.0
    xb = bf16(x)
    q, sf, normed, _ = call(xb, None, torch.ones(512, device="cuda"), 1e-12)
    want_q, want_sf = oracle.cast_to_fp8(xb.view(torch.int16).cpu().numpy().view(np.uint16))
    assert np.array_equal(q, want_q) and np.array_equal(sf, want_sf)
    assert np.array_equal(normed, xb.view(torch.int16).cpu().numpy().view(np.uint16))


def test_many_rows_past_2_to_32_bytes():
    """2^25 + 7 rows of 128: offsets past 32 bits and more rows than one launch takes; rows are those of a call on them alone."""
    R, C = 2 ** 25 + 7, 128
    x = torch.empty(R, C, dtype=torch.bfloat16, device="cuda")
    x.view(torch.int16).random_(0, 0x4200)                      # every finite magnitude up to 2^5
    w = torch.ones(C, device="cuda")
    q = torch.empty(R, C, dtype=torch.uint8, device="cuda")
    sf = torch.empty(R, 4, dtype=torch.uint8, device="cuda")
    moe.moe_rmsnorm_to_fp8(q, sf, None, None, x, None, w, moe.MOE_F32, R, C, 1e-6)
    torch.cuda.synchronize()
    for at in (0, 2 ** 23 - 2, 2 ** 24 - 3, R - 5):
        part = x[at:at + 5].clone()
        got = call(part, None, w, 1e-6, normed=False, out=False)
        assert np.array_equal(q[at:at + 5].cpu().numpy(), got[0]) and np.array_equal(sf[at:at + 5].cpu().numpy(), got[1])
    check(got, part, None, w, 1e-6)
    del x, q, sf
    torch.cuda.empty_cache()
