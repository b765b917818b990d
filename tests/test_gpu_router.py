"""GPU parity of the top-k router against the fp64 oracle: ids exactly, weights within the
rounding of an FP32 softmax.

Tolerance of a weight e_j / sum * scale, with u = 2^-24 and D = the largest distance m - x whose
exponential is not negligible (at most 104, below which FP32 exp is zero): the difference x - m
rounds by u*D absolutely, which is u*D relative in exp; exp itself is within 2 ulp (4u); the sum of n
positive terms adds (n - 1) u on top of its terms' own error; the division and the scaling round
by u each: 2 * (D + 4) u + n u + 2u relative, and 2^-126 absolute for flushed subnormals."""
import math

import numpy as np
import pytest
import torch

from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

import block_scaled_fp8_dispatch_amd as moe  # noqa: E402
import oracle  # noqa: E402


def run(logits, k, over_all, scale=1.0):
    T, E = logits.shape
    idx = torch.full((T + 1, k), -77, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), -7.0, device="cuda")
    ty = moe.MOE_BF16 if logits.dtype == torch.bfloat16 else moe.MOE_F32
    over = moe.MOE_ROUTER_SOFTMAX_ALL if over_all else moe.MOE_ROUTER_SOFTMAX_CHOSEN
    moe.moe_topk_router(idx, w, logits, ty, T, E, k, over, scale)
    torch.cuda.synchronize()
    assert (idx[T] == -77).all() and (w[T] == -7.0).all(), "a store went past the last token"
    return idx[:T].cpu().numpy(), w[:T].double().cpu().numpy()


def check(logits, k, over_all, scale=1.0):
    print(f"[router] {tuple(logits.shape)} {logits.dtype} k={k} all={over_all}", flush=True)
    idx, w = run(logits, k, over_all, scale)
    x = logits.double().cpu().numpy()
    ref_idx, ref_w = oracle.topk_router(x, k, over_all, scale)
    assert np.array_equal(idx, ref_idx)
    fin = np.isfinite(x)
    spread = float(np.maximum(np.where(fin, x, -np.inf).max(1) - np.where(fin, x, np.inf).min(1), 0.0).max())
    u = 2.0 ** -24
    tol = (2 * (min(spread, 104.0) + 4) + x.shape[1] + 2) * u
    assert (np.abs(w - ref_w) <= tol * np.abs(ref_w) + abs(scale) * 2.0 ** -126).all(), np.abs(w - ref_w).max()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 4, 2), (5, 8, 8), (64, 32, 8), (257, 33, 7), (100, 64, 6), (65, 128, 5),
                                   (33, 161, 6), (9, 256, 8), (7, 511, 64), (5, 1024, 64), (1000, 16, 3), (2, 65, 64),
                                   (31, 2, 1), (130, 12, 12)])
@pytest.mark.parametrize("over_all", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_random(T, E, k, over_all, dtype):
    g = torch.Generator(device="cuda").manual_seed(T * 1000 + E)
    x = (torch.randn(T, E, generator=g, device="cuda") * 3).to(dtype)
    check(x, k, over_all, 2.5)


@pytest.mark.parametrize("E", [6, 40, 70, 300])
@pytest.mark.parametrize("over_all", [False, True])
def test_ties_masks_and_extremes(E, over_all):
    low = torch.finfo(torch.float32).min
    inf, nan = math.inf, math.nan
    x = torch.zeros(14, E)
    x[1] = low                               # masked by the type's lowest value: still a choice
    x[2] = -inf                              # nothing left
    x[3] = nan
    x[4] = -inf
    x[4, E - 1] = -5.0                       # one left
    x[5, ::2], x[5, 1::2] = -0.0, 0.0        # equal values
    x[6] = torch.arange(E) % 3               # ties
    x[7] = -torch.arange(E).float()
    x[8] = inf
    x[9, 2], x[9, E - 2] = inf, inf
    x[10] = torch.where(torch.arange(E) % 2 == 0, torch.tensor(nan), torch.arange(E).float() / 8)
    x[11] = 1e-42 * torch.arange(E)          # subnormal logits
    x[12] = low
    x[12, 1] = 3e38
    x[13] = torch.arange(E).float() * 40     # exponentials that underflow
    for k in (1, 3, 6):
        check(x.cuda(), k, over_all)
    check(x.to(torch.bfloat16).cuda(), 5, over_all, -1.0)


@pytest.mark.parametrize("E", [8, 24, 60, 100, 256, 300, 1000])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_neighbours_in_the_last_bits(E, sign):
    """Logits that differ only in their last bits, among the chosen and at the border, next to tokens
    whose logits end in zero bits, in every order."""
    g = torch.Generator().manual_seed(E)
    rows = []
    for spread in (1, 2, 7, 300):                       # steps of 2^-23 between neighbours
        v = 1.0 + torch.randperm(E, generator=g).float() * spread * 2.0 ** -23
        rows += [v, torch.where(torch.rand(E, generator=g) < 0.3, v, torch.ones(E)), v.round()]
    v = torch.randn(E, generator=g)
    v[torch.randperm(E, generator=g)[: min(5, E - 2)]] = 3.0 + torch.arange(min(5, E - 2)).float() * 2.0 ** -22
    rows += [v, torch.randn(E, generator=g).to(torch.bfloat16).float(), torch.zeros(E)]
    x = (torch.stack(rows) * sign).cuda()
    for k in (1, 4, 8):
        check(x, k, False)
    if E >= 24:
        check(x, 16, True)
        check(x, 17, True)


def test_many_tokens_and_graph():
    g = torch.Generator(device="cuda").manual_seed(5)
    xs = [torch.randn(4097, 32, generator=g, device="cuda") for _ in range(3)]
    eager = [run(x, 8, False) for x in xs]
    buf = xs[0].clone()
    idx = torch.empty(4097, 8, dtype=torch.int32, device="cuda")
    w = torch.empty(4097, 8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_topk_router(idx, w, buf, moe.MOE_F32, 4097, 32, 8, moe.MOE_ROUTER_SOFTMAX_CHOSEN)
    for i in (0, 1, 2, 0):
        buf.copy_(xs[i])
        idx.fill_(-9)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(idx.cpu().numpy(), eager[i][0])
        assert np.array_equal(w.double().cpu().numpy(), eager[i][1])
    ref_idx, _ = oracle.topk_router(xs[0].double().cpu().numpy(), 8, False)
    assert np.array_equal(eager[0][0], ref_idx)
