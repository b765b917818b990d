"""GPU parity of the 4-bit casts against the oracle: every code, scale byte and value bit for bit (nothing rounds before the
decision, and the cast back is exact), at sizes from one block to several launches' worth of rows."""
import numpy as np
import pytest
import torch

from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

import block_scaled_fp8_dispatch_amd as moe  # noqa: E402
import oracle  # noqa: E402

TYPES = {moe.MOE_BF16: torch.bfloat16, moe.MOE_F32: torch.float32}


def cast(x, ty, guard=256):
    """codes, scale bytes of x [R, C]; what lies behind both outputs must stay."""
    R, C = x.shape
    q = torch.full((R * C // 2 + guard,), 0xA5, dtype=torch.uint8, device="cuda")
    sf = torch.full((R * C // 32 + guard,), 0xA5, dtype=torch.uint8, device="cuda")
    moe.moe_cast_to_fp4(x, ty, R, C, q, sf)
    torch.cuda.synchronize()
    assert (q[R * C // 2:] == 0xA5).all() and (sf[R * C // 32:] == 0xA5).all(), "a store went past the end"
    return q[: R * C // 2].view(R, C // 2), sf[: R * C // 32].view(R, C // 32)


def back(q, sf, ty, guard=64):
    R, C = q.shape[0], 2 * q.shape[1]
    x = torch.full((R * C + guard,), 7.0, dtype=TYPES[ty], device="cuda")
    moe.moe_cast_from_fp4(q, sf, R, C, x, ty)
    torch.cuda.synchronize()
    assert (x[R * C:] == 7.0).all(), "a store went past the end"
    return x[: R * C].view(R, C)


def edges(C, seed):
    """Rows of ties, boundaries of the scale rule, subnormals, signed zeros and the largest numbers."""
    rng = np.random.default_rng(seed)
    rows = [rng.standard_normal(C), rng.integers(-48, 49, C) / 8.0, np.zeros(C), -np.zeros(C), rng.standard_normal(C) * 1e-39,
            rng.standard_normal(C) * 2.0 ** -126, np.full(C, 3.38e38), rng.integers(-2, 3, C) * 1e-45,
            6.0 * 2.0 ** rng.integers(-120, 120, C), -6.03125 * 2.0 ** rng.integers(-120, 120, C)]
    for j in range(0, C, 32):
        rows[1][j] = 6.0                                        # the block's scale is 1: eighths are its ties
    return np.array(rows, dtype=np.float32)


@pytest.mark.parametrize("ty", list(TYPES))
@pytest.mark.parametrize("R,C", [(1, 32), (3, 32), (1, 128), (7, 96), (33, 2048), (129, 1056), (5, 18432), (2051, 64)])
def test_cast(R, C, ty):
    print(f"[fp4] cast {R} {C} {ty}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(R + C)
    x = torch.randn(R, C, generator=g, device="cuda") * torch.exp2(torch.randint(-20, 20, (R, C), generator=g, device="cuda").float())
    x = x.to(TYPES[ty])
    q, sf = cast(x, ty)
    want_q, want_sf = oracle.cast_to_fp4(x.double().cpu().numpy())
    assert np.array_equal(sf.cpu().numpy(), want_sf) and np.array_equal(q.cpu().numpy(), want_q)
    v = back(q, sf, ty)
    assert np.array_equal(v.double().cpu().numpy(), oracle.cast_from_fp4(want_q, want_sf))


@pytest.mark.parametrize("ty", list(TYPES))
def test_cast_edges(ty):
    x = torch.from_numpy(edges(160, 3)).cuda().to(TYPES[ty])
    q, sf = cast(x, ty)
    want_q, want_sf = oracle.cast_to_fp4(x.double().cpu().numpy())
    assert np.array_equal(sf.cpu().numpy(), want_sf) and np.array_equal(q.cpu().numpy(), want_q)


@pytest.mark.parametrize("ty", list(TYPES))
def test_infinities_and_nan_stay_in_their_block(ty):
    x = torch.randn(4, 256, device="cuda").to(TYPES[ty])
    q0, sf0 = cast(x, ty)
    x[0, 5], x[1, 64], x[3, 255] = float("inf"), float("nan"), -float("inf")
    q, sf = cast(x, ty)
    hit = torch.zeros(4, 8, dtype=torch.bool, device="cuda")
    hit[0, 0] = hit[1, 2] = hit[3, 7] = True
    assert (sf[hit] == 255).all() and torch.equal(sf[~hit], sf0[~hit])
    blocks, blocks0 = q.view(4, 8, 16), q0.view(4, 8, 16)
    assert (blocks[hit] == 0).all() and torch.equal(blocks[~hit], blocks0[~hit])
    v = back(q, sf, ty).view(4, 8, 32)
    assert torch.isnan(v[hit]).all() and torch.isfinite(v[~hit]).all()


@pytest.mark.parametrize("ty", list(TYPES))
def test_every_code_at_every_scale(ty):
    """All 16 codes at all 256 scale bytes: the exact number, rounded to the type once (subnormal bf16 and FP32 numbers, and
    infinities at the top, included)."""
    q = torch.arange(256, device="cuda").view(1, 256).repeat(256, 1).to(torch.uint8)         # every pair of codes
    sf = torch.arange(256, device="cuda").view(256, 1).repeat(1, 16).to(torch.uint8)
    v = back(q, sf, ty)
    with np.errstate(over="ignore"):
        want = torch.from_numpy(oracle.cast_from_fp4(q.cpu().numpy(), sf.cpu().numpy())).to(TYPES[ty]).cuda()
    ok = (v == want) & (torch.signbit(v) == torch.signbit(want)) | torch.isnan(v) & torch.isnan(want)
    assert ok.all(), torch.nonzero(~ok)[:4]


def test_weights_cast_here_pack_and_multiply_like_the_generators():
    """The cast's output is what the packing reads: the same bytes as the CPU quantiser's of the same numbers."""
    from synth.generate import cast_fp4_blocks
    g = torch.Generator().manual_seed(5)
    w = torch.randn(272, 384, generator=g) * 0.02
    want_q, want_sf = cast_fp4_blocks(w)
    q, sf = cast(w.cuda(), moe.MOE_F32)
    assert torch.equal(q.cpu(), want_q) and torch.equal(sf.cpu(), want_sf)
    packed = [torch.empty(moe.moe_gemm_packed_b_bytes(1, 272, 384), dtype=torch.uint8, device="cuda") for _ in range(2)]
    moe.moe_gemm_prepare_b(1, 272, 384, q, sf, packed[0])
    moe.moe_gemm_prepare_b(1, 272, 384, want_q.cuda(), want_sf.cuda(), packed[1])
    assert torch.equal(packed[0], packed[1])


def test_past_2_to_32_elements():
    """5 * 2^30 bf16 elements: offsets past 32 bits; the last rows are those of a call on them alone."""
    R, C = 5 * 2 ** 18, 4096
    x = torch.empty(R, C, dtype=torch.bfloat16, device="cuda")
    x.view(torch.int16).random_(-0x4200, 0x4200)                # magnitudes of every kind, NaN among them
    x[-1, 7] = 1000.0
    q = torch.empty(R, C // 2, dtype=torch.uint8, device="cuda")
    sf = torch.empty(R, C // 32, dtype=torch.uint8, device="cuda")
    moe.moe_cast_to_fp4(x, moe.MOE_BF16, R, C, q, sf)
    for rows in (slice(0, 5), slice(R // 2 - 2, R // 2 + 3), slice(R - 5, R)):
        one = x[rows].clone()
        a, b = cast(one, moe.MOE_BF16)
        assert torch.equal(q[rows], a) and torch.equal(sf[rows], b)
    want_q, want_sf = oracle.cast_to_fp4(x[-2:].double().cpu().numpy())
    assert np.array_equal(q[-2:].cpu().numpy(), want_q) and np.array_equal(sf[-2:].cpu().numpy(), want_sf)
    x.fill_(9.0)
    moe.moe_cast_from_fp4(q, sf, R, C, x, moe.MOE_BF16)
    # (a block whose largest number rounds up to 2^128 holds an infinity in bf16)
    want = torch.from_numpy(oracle.cast_from_fp4(want_q, want_sf)).to(torch.bfloat16)
    assert torch.allclose(x[-2:].cpu(), want, rtol=0, atol=0, equal_nan=True)
    assert torch.equal(x[R // 2].view(torch.int16), back(q[R // 2:R // 2 + 1], sf[R // 2:R // 2 + 1], moe.MOE_BF16)[0].view(torch.int16))
    del x, q, sf
    torch.cuda.empty_cache()
