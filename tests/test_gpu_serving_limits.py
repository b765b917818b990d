"""The router, the few-token forward and the FP8 x FP8 GEMMs at their documented limits: data past 4 GiB, two calls
at once on streams with a workspace each, captured calls whose device-side counts and groups change
between replays. Tolerances as in test_gpu_router.py and test_gpu_fp8_gemm.py."""
import numpy as np
import pytest
import torch

from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

import block_scaled_fp8_dispatch_amd as moe  # noqa: E402
import oracle  # noqa: E402
from test_gpu_fp8_gemm import POISON, Problem, alignment_bound, make  # noqa: E402


def gpu_codes(*shape):
    """e4m3 codes without NaN."""
    return torch.randint(0, 0x7F, shape, dtype=torch.uint8, device="cuda")


def gemm_buffers(rows, G, n, ty):
    ws = torch.empty(moe.moe_fp8_gemm_workspace_bytes(rows, G), dtype=torch.uint8, device="cuda")
    d = torch.full((rows, n), POISON[ty], dtype=torch.int32 if ty == moe.MOE_F32 else torch.int16, device="cuda")
    return ws, d


def check_rows(d, rows, a, a_sf, b, b_sf, K, ty):
    got = d[torch.tensor(rows, device="cuda")].cpu().numpy()
    args = (a[rows].cpu().numpy(), a_sf[rows].cpu().numpy(), b.cpu().numpy(), b_sf.cpu().numpy(), K)
    ref = oracle.fp8_gemm(*args)
    if ty == moe.MOE_F32:
        ok = oracle.gemm_f32_within_bound(got.view(np.float32), ref["exact"], ref["bound"])
    else:
        ok = oracle.gemm_bf16_within_bound(got.view(np.uint16), ref["exact"], ref["bound"] + alignment_bound(*args))
    assert ok.all(), np.argwhere(~ok)[:4]


@pytest.mark.parametrize("M,N,K,ty", [
    (524287, 96, 8192, moe.MOE_BF16),      # A of 4 GiB less one row
    (60001, 40001, 128, moe.MOE_BF16),     # D of 4.5 GiB, rows at every alignment
    (40000, 40008, 128, moe.MOE_F32),      # D of 6 GiB
    (20, 1100001, 128, moe.MOE_F32),       # few rows, many columns
])
def test_dense_past_4gb(M, N, K, ty):
    print(f"[limits] dense {M} {N} {K} {ty}", flush=True)
    a, b = gpu_codes(M, K), gpu_codes(N, K)
    a_sf = torch.randint(121, 134, (M, 4 * -(-K // 512)), dtype=torch.uint8, device="cuda")
    b_sf = torch.randint(121, 134, (-(-N // 128), 4 * -(-K // 512)), dtype=torch.uint8, device="cuda")
    ws, d = gemm_buffers(M, 1, N, ty)
    moe.moe_fp8_gemm(d, ty, a, a_sf, M, N, K, b, b_sf, ws)
    torch.cuda.synchronize()
    check_rows(d, [0, M // 2, M - 1], a, a_sf, b, b_sf, K, ty)
    del a, b, d
    torch.cuda.empty_cache()


def test_router_past_4gb():
    """Logits of 4.5 GiB: the last tokens' choice and weights are those of a call on them alone."""
    T, E, k = 1179650, 1024, 4
    x = torch.randn(T, E, device="cuda")
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    moe.moe_topk_router(idx, w, x, moe.MOE_F32, T, E, k, moe.MOE_ROUTER_SOFTMAX_CHOSEN)
    n = 40
    last_idx, last_w = torch.empty(n, k, dtype=torch.int32, device="cuda"), torch.empty(n, k, device="cuda")
    moe.moe_topk_router(last_idx, last_w, x[-n:].clone(), moe.MOE_F32, n, E, k, moe.MOE_ROUTER_SOFTMAX_CHOSEN)
    torch.cuda.synchronize()
    assert torch.equal(idx[-n:], last_idx) and torch.equal(w[-n:], last_w)
    assert (idx >= 0).all()
    ref_idx, _ = oracle.topk_router(x[-n:].double().cpu().numpy(), k, False)
    assert np.array_equal(last_idx.cpu().numpy(), ref_idx)
    del x, idx, w
    torch.cuda.empty_cache()


def test_two_streams_at_once():
    """Calls on two streams, each with a workspace of its own, give what they give one after another."""
    K, N, G = 512, 520, 3
    grp = torch.randint(-1, G, (900,), dtype=torch.int32, device="cuda")
    cnt = torch.tensor([300, 7, 0], dtype=torch.int32, device="cuda")
    probs = [Problem(900, N, K, G, moe.MOE_BF16, seed=s) for s in (1, 2)]

    def call(p, contiguous):
        a, a_sf, b, b_sf = p.dev
        if contiguous:
            moe.moe_m_grouped_fp8_gemm_contiguous(p.d, p.d_type, a, a_sf, grp, 900, G, N, K, b, b_sf, p.ws)
        else:
            moe.moe_m_grouped_fp8_gemm_masked(p.d, p.d_type, a, a_sf, cnt, G, 300, 100, N, K, b, b_sf, p.ws)

    want = []
    for p, contiguous in zip(probs, (True, False)):
        p.d.fill_(POISON[p.d_type])
        call(p, contiguous)
        torch.cuda.synchronize()
        want.append(p.d.clone())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for p in probs:
        p.d.fill_(POISON[p.d_type])
    torch.cuda.synchronize()
    for _ in range(20):
        for p, s, contiguous in zip(probs, streams, (True, False)):
            with torch.cuda.stream(s):
                call(p, contiguous)
    torch.cuda.synchronize()
    for p, w in zip(probs, want):
        assert torch.equal(p.d, w)


@pytest.mark.parametrize("M", [600, 20000])          # grouped in one launch, and in several
def test_captured_groups_and_counts_change(M):
    K, N, G, max_m = 256, 264, 5, 120
    ha, ha_sf, hb, hb_sf = make(M, N, K, G, seed=M)
    a, a_sf, b, b_sf = (torch.from_numpy(v).cuda() for v in (ha, ha_sf, hb, hb_sf))
    ws, d = gemm_buffers(M, G, N, moe.MOE_BF16)
    ws2, d2 = gemm_buffers(G * max_m, G, N, moe.MOE_BF16)
    grp = torch.zeros(M, dtype=torch.int32, device="cuda")
    cnt = torch.zeros(G, dtype=torch.int32, device="cuda")

    def calls():
        moe.moe_m_grouped_fp8_gemm_contiguous(d, moe.MOE_BF16, a, a_sf, grp, M, G, N, K, b, b_sf, ws)
        moe.moe_m_grouped_fp8_gemm_masked(d2, moe.MOE_BF16, a, a_sf, cnt, G, max_m, 64, N, K, b, b_sf, ws2)

    gen = torch.Generator(device="cuda").manual_seed(M)
    grps = [torch.randint(-1, G + 1, (M,), generator=gen, dtype=torch.int32, device="cuda"),
            torch.full((M,), -1, dtype=torch.int32, device="cuda"), torch.full((M,), 2, dtype=torch.int32, device="cuda")]
    cnts = [torch.randint(-1, max_m + 9, (G,), generator=gen, dtype=torch.int32, device="cuda"),
            torch.zeros(G, dtype=torch.int32, device="cuda"), torch.full((G,), max_m, dtype=torch.int32, device="cuda")]

    def eager(i):
        grp.copy_(grps[i])
        cnt.copy_(cnts[i])
        d.fill_(POISON[moe.MOE_BF16])
        d2.fill_(POISON[moe.MOE_BF16])
        calls()
        torch.cuda.synchronize()
        return d.clone(), d2.clone()

    want = [eager(i) for i in range(3)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for i in (0, 1, 2, 0, 2):
        grp.copy_(grps[i])
        cnt.copy_(cnts[i])
        d.fill_(POISON[moe.MOE_BF16])
        d2.fill_(POISON[moe.MOE_BF16])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d, want[i][0]) and torch.equal(d2, want[i][1]), i


@pytest.mark.parametrize("ty", [moe.MOE_BF16, moe.MOE_F32])
@pytest.mark.parametrize("M,N,K", [(1000, 2000, 2048), (513, 1031, 2176), (65, 4099, 1024), (300, 640, 1152), (17, 5000, 1280),
                                   (97, 2311, 384), (33, 7168, 2048), (15, 31, 7168)])
def test_few_or_small_tiles(M, N, K, ty):
    """Products between the smallest and a round of large tiles, ragged both ways, whole K shares and not."""
    print(f"[limits] dense {M} {N} {K} {ty}", flush=True)
    p = Problem(M, N, K, 1, ty, seed=M)
    d = p.dense()
    p.check(d, np.unique(np.r_[0:min(M, 40), M // 2, M - 1 - np.arange(min(M, 20))]))
    assert np.array_equal(p.dense(), d)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E", [33, 36, 63, 64, 100, 127, 128, 201, 252, 256, 257, 384, 510, 512, 644, 1023, 1024])
def test_router_rows_end_anywhere(E, dtype):
    """Expert counts around the kernels' borders, multiples of 4 (loaded in fours) and not; the row behind
    the last token would win every choice."""
    T, k = 300, 8
    x = torch.full((T + 1, E), 1e30, device="cuda", dtype=dtype)
    x[:T] = torch.randn(T, E, device="cuda").to(dtype)
    idx = torch.full((T + 1, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), -7.0, device="cuda")
    moe.moe_topk_router(idx, w, x, moe.MOE_BF16 if dtype == torch.bfloat16 else moe.MOE_F32, T, E, k, moe.MOE_ROUTER_SOFTMAX_ALL)
    torch.cuda.synchronize()
    ref_idx, ref_w = oracle.topk_router(x[:T].double().cpu().numpy(), k, True)
    assert np.array_equal(idx[:T].cpu().numpy(), ref_idx)
    # |x| < 6: distances below 12; the rounding of test_gpu_router.py at D = 12
    tol = (2 * (12 + 4) + E + 2) * 2.0 ** -24
    assert (np.abs(w[:T].double().cpu().numpy() - ref_w) <= tol * ref_w + 2.0 ** -126).all()
    assert (idx[T] == -7).all() and (w[T] == -7.0).all()


@pytest.mark.parametrize("E", [30, 64, 250, 256])
def test_router_passes(E):
    """More tokens than one pass of the grid takes: as calls on parts that one pass takes."""
    T, k, part = 100003, 8, 20000
    x = torch.randn(T, E, device="cuda")
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    moe.moe_topk_router(idx, w, x, moe.MOE_F32, T, E, k, moe.MOE_ROUTER_SOFTMAX_CHOSEN)
    for a in range(0, T, part):
        xs = x[a:a + part].clone()
        n = xs.shape[0]
        i2, w2 = torch.empty(n, k, dtype=torch.int32, device="cuda"), torch.empty(n, k, device="cuda")
        moe.moe_topk_router(i2, w2, xs, moe.MOE_F32, n, E, k, moe.MOE_ROUTER_SOFTMAX_CHOSEN)
        torch.cuda.synchronize()
        assert torch.equal(idx[a:a + part], i2) and torch.equal(w[a:a + part], w2)


@pytest.mark.parametrize("M,G", [(1024, 256), (1025, 256), (1024, 257), (257, 256), (1000, 3), (16385, 2), (4097, 5), (8193, 5)])
def test_contiguous_grouping_borders(M, G):
    """Row and group counts at which the grouping changes its kernel."""
    K, N = 128, 40
    p = Problem(M, N, K, G, moe.MOE_BF16, seed=M + G)
    grp = np.random.default_rng(G).integers(-1, G, size=M).astype(np.int32)
    grp[0] = G - 1
    d = p.contiguous(grp)
    for g in range(0, G, max(1, G // 20)):
        p.check(d, np.nonzero(grp == g)[0], g)
    p.check(d, np.nonzero(grp == G - 1)[0], G - 1)
    assert (d[grp < 0] == POISON[moe.MOE_BF16]).all()
    assert np.array_equal(p.contiguous(grp), d), "two calls gave different bytes"
