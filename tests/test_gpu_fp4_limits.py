"""The norm with FP8 output, the 4-bit casts and the FP4 x FP4 GEMMs at their documented limits: data past 4 GiB, two calls at
once on streams with a workspace each, captured calls whose device-side counts and groups change between replays, and a run of
them together as a layer uses them. Tolerances as in the tests of each."""
import numpy as np
import pytest
import torch

from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

import block_scaled_fp8_dispatch_amd as moe  # noqa: E402
import oracle  # noqa: E402
from test_gpu_fp4_gemm import POISON, Problem, make, pack  # noqa: E402
from test_gpu_rmsnorm import check as check_norm  # noqa: E402


def gpu_codes(rows, K):
    return (torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device="cuda"),
            torch.randint(121, 134, (rows, K // 32), dtype=torch.uint8, device="cuda"))


def buffers(rows, G, n, ty):
    ws = torch.empty(moe.moe_fp4_gemm_workspace_bytes(rows, G), dtype=torch.uint8, device="cuda")
    d = torch.full((rows, n), POISON[ty], dtype=torch.int32 if ty == moe.MOE_F32 else torch.int16, device="cuda")
    return ws, d


def check_rows(got, a, a_sf, b, b_sf, K, ty):
    ref = oracle.fp4_gemm(a.cpu().numpy(), a_sf.cpu().numpy(), b.cpu().numpy(), b_sf.cpu().numpy(), K)
    got = got.cpu().numpy()
    if ty == moe.MOE_F32:
        ok = oracle.gemm_f32_within_bound(got.view(np.float32), ref["exact"], ref["bound"])
    else:
        ok = oracle.gemm_bf16_within_bound(got.view(np.uint16), ref["exact"], ref["bound"])
    assert ok.all(), np.argwhere(~ok)[:4]


@pytest.mark.parametrize("M,N,K,ty", [
    (524287, 96, 8192, moe.MOE_BF16),      # A of 2 GiB less one row: rows times K at its limit
    (60001, 40000, 128, moe.MOE_BF16),     # D of 4.5 GiB
    (40000, 40016, 128, moe.MOE_F32),      # D of 6 GiB
    (20, 1100000, 128, moe.MOE_F32),       # few rows, many columns
    (3, 16, 2 ** 22, moe.MOE_F32),         # the longest sums
])
def test_dense_past_4gb(M, N, K, ty):
    print(f"[limits] fp4 dense {M} {N} {K} {ty}", flush=True)
    a, a_sf = gpu_codes(M, K)
    b, b_sf = gpu_codes(N, K)
    packed = pack(b, b_sf, N, K, 1)
    ws, d = buffers(M, 1, N, ty)
    moe.moe_fp4_gemm(d, ty, a, a_sf, M, N, K, packed, ws)
    torch.cuda.synchronize()
    rows = torch.tensor(sorted({0, 1, M // 2, M - 2, M - 1}), device="cuda")
    check_rows(d[rows], a[rows], a_sf[rows], b, b_sf, K, ty)
    del a, b, d, packed
    torch.cuda.empty_cache()


def test_b_beyond_4gb():
    """Packed B above 4 GiB: the last groups lie past 32-bit byte offsets from its start."""
    G, N, K = 300, 4096, 7168
    b, b_sf = gpu_codes(G * N, K)
    packed = pack(b, b_sf, N, K, G)
    assert packed.numel() > 2 ** 32
    for rows, em in ((3, 3), (300, 300)):                         # one row tile a group, and several
        a, a_sf = gpu_codes(G * rows, K)
        cnt = torch.full((G,), rows - 1, dtype=torch.int32, device="cuda")
        ws, d = buffers(G * rows, G, N, moe.MOE_BF16)
        moe.moe_m_grouped_fp4_gemm_masked(d, moe.MOE_BF16, a, a_sf, cnt, G, rows, em, N, K, packed, ws)
        torch.cuda.synchronize()
        for g in (0, 150, 296, 299):
            at = slice(g * rows, (g + 1) * rows - 1)
            check_rows(d[at][:4], a[at][:4], a_sf[at][:4], b[g * N:(g + 1) * N], b_sf[g * N:(g + 1) * N], K, moe.MOE_BF16)
            assert (d[(g + 1) * rows - 1] == POISON[moe.MOE_BF16]).all()
        del a, d
    del b, packed
    torch.cuda.empty_cache()


def test_two_streams_at_once():
    """Calls on two streams, each with a workspace of its own, give what they give one after another."""
    K, N, G = 512, 528, 3
    grp = torch.randint(-1, G, (900,), dtype=torch.int32, device="cuda")
    cnt = torch.tensor([300, 7, 0], dtype=torch.int32, device="cuda")
    probs = [Problem(900, N, K, G, moe.MOE_BF16, seed=s) for s in (1, 2)]

    def call(p, contiguous):
        if contiguous:
            moe.moe_m_grouped_fp4_gemm_contiguous(p.d, p.d_type, p.ga, p.ga_sf, grp, 900, G, N, K, p.packed, p.ws)
        else:
            moe.moe_m_grouped_fp4_gemm_masked(p.d, p.d_type, p.ga, p.ga_sf, cnt, G, 300, 100, N, K, p.packed, p.ws)

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
    K, N, G, max_m = 256, 272, 5, 120
    ha, ha_sf, hb, hb_sf = make(M, N, K, G, seed=M)
    a, a_sf, b, b_sf = (torch.from_numpy(v).cuda() for v in (ha, ha_sf, hb, hb_sf))
    packed = pack(b, b_sf, N, K, G)
    ws, d = buffers(M, G, N, moe.MOE_BF16)
    ws2, d2 = buffers(G * max_m, G, N, moe.MOE_F32)
    grp = torch.zeros(M, dtype=torch.int32, device="cuda")
    cnt = torch.zeros(G, dtype=torch.int32, device="cuda")

    def calls():
        moe.moe_m_grouped_fp4_gemm_contiguous(d, moe.MOE_BF16, a, a_sf, grp, M, G, N, K, packed, ws)
        moe.moe_m_grouped_fp4_gemm_masked(d2, moe.MOE_F32, a, a_sf, cnt, G, max_m, 64, N, K, packed, ws2)

    gen = torch.Generator(device="cuda").manual_seed(M)
    grps = [torch.randint(-1, G + 1, (M,), generator=gen, dtype=torch.int32, device="cuda"),
            torch.full((M,), -1, dtype=torch.int32, device="cuda"), torch.full((M,), 2, dtype=torch.int32, device="cuda")]
    cnts = [torch.randint(-1, max_m + 9, (G,), generator=gen, dtype=torch.int32, device="cuda"),
            torch.zeros(G, dtype=torch.int32, device="cuda"), torch.full((G,), max_m, dtype=torch.int32, device="cuda")]

    def eager(i):
        grp.copy_(grps[i])
        cnt.copy_(cnts[i])
        d.fill_(POISON[moe.MOE_BF16])
        d2.fill_(POISON[moe.MOE_F32])
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
        d2.fill_(POISON[moe.MOE_F32])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d, want[i][0]) and torch.equal(d2, want[i][1]), f"replay {i}"
        assert all(torch.equal(x, y) for x, y in zip(eager((i + 1) % 3), want[(i + 1) % 3]))


class Layer:
    """Hidden states and residual -> norm -> the gate's FP8 product and a 4-bit projection of the normed rows, with weights
    that were cast and packed on the GPU."""

    def __init__(self, T, H, N, E, seed):
        self.T, self.H, self.N, self.E = T, H, N, E
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.weight = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
        w = torch.randn(N, H, generator=g, device="cuda") * 0.02
        self.b = torch.empty(N, H // 2, dtype=torch.uint8, device="cuda")
        self.b_sf = torch.empty(N, H // 32, dtype=torch.uint8, device="cuda")
        moe.moe_cast_to_fp4(w, moe.MOE_F32, N, H, self.b, self.b_sf)
        self.packed = pack(self.b, self.b_sf, N, H, 1)
        self.gate = torch.randint(0, 0x30, (E, H), generator=g, dtype=torch.uint8, device="cuda")
        self.gate_sf = torch.full((-(-E // 128), 4 * -(-H // 512)), 123, dtype=torch.uint8, device="cuda")
        u8 = lambda *s: torch.empty(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.x8, self.x8_sf, self.x4, self.x4_sf = u8(T, H), u8(T, 4 * -(-H // 512)), u8(T, H // 2), u8(T, H // 32)
        self.normed = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        self.logits = torch.empty(T, E, device="cuda")
        self.z = torch.empty(T, N, dtype=torch.int16, device="cuda")
        self.ws = u8(moe.moe_gemm_workspace_bytes(T, 1))

    def __call__(self, x, residual, stream=None):
        """residual is updated in place."""
        T, H = self.T, self.H
        moe.moe_rmsnorm_to_fp8(self.x8, self.x8_sf, self.normed, residual, x, residual, self.weight, moe.MOE_BF16, T, H, 1e-5,
                               stream=stream)
        moe.moe_fp8_gemm(self.logits, moe.MOE_F32, self.x8, self.x8_sf, T, self.E, H, self.gate, self.gate_sf, self.ws, stream=stream)
        moe.moe_cast_to_fp4(self.normed, moe.MOE_BF16, T, H, self.x4, self.x4_sf, stream=stream)
        moe.moe_fp4_gemm(self.z, moe.MOE_BF16, self.x4, self.x4_sf, T, self.N, H, self.packed, self.ws, stream=stream)

    def outputs(self, residual):
        torch.cuda.synchronize()
        return [t.view(torch.uint8).cpu().numpy() for t in (self.x8, self.x8_sf, self.normed, self.logits, self.x4, self.x4_sf, self.z, residual)]

    def poison(self):
        for t in (self.x8, self.x8_sf, self.normed, self.logits, self.x4, self.x4_sf, self.z, self.ws):
            t.view(torch.uint8).fill_(0x7F)


def test_a_layer():
    T, H, N, E = 37, 640, 272, 24
    layer = Layer(T, H, N, E, seed=2)
    g = torch.Generator(device="cuda").manual_seed(3)
    xs = [torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3)]
    rs = [(3 * torch.randn(T, H, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(3)]
    eager = []
    for x, r in zip(xs, rs):
        layer.poison()
        r = r.clone()
        layer(x, r)
        eager.append(layer.outputs(r))
    layer.poison()
    r = rs[0].clone()
    layer(xs[0], r)
    torch.cuda.synchronize()
    host = lambda t: t.cpu().numpy()  # noqa: E731
    bits = lambda t: host(t.view(torch.int16)).view(np.uint16)  # noqa: E731
    check_norm((host(layer.x8), host(layer.x8_sf), bits(layer.normed), bits(r)), xs[0], rs[0], layer.weight, 1e-5)
    ref = oracle.fp8_gemm(host(layer.x8), host(layer.x8_sf), host(layer.gate), host(layer.gate_sf), H)
    assert oracle.gemm_f32_within_bound(host(layer.logits), ref["exact"], ref["bound"]).all()
    q, sf = oracle.cast_to_fp4(oracle.bf16_bits_to_f64(bits(layer.normed)))
    assert np.array_equal(host(layer.x4), q) and np.array_equal(host(layer.x4_sf), sf)
    check_rows(layer.z, layer.x4, layer.x4_sf, layer.b, layer.b_sf, H, moe.MOE_BF16)

    # on another stream than the current one
    side = torch.cuda.Stream()
    layer.poison()
    r = rs[1].clone()
    side.wait_stream(torch.cuda.current_stream())
    layer(xs[1], r, stream=side)
    assert all(np.array_equal(a, b) for a, b in zip(layer.outputs(r), eager[1]))

    # captured once, replayed with new activations between eager calls
    x, r = xs[0].clone(), rs[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(x, r)
    for i in (0, 1, 2, 1, 0):
        x.copy_(xs[i])
        r.copy_(rs[i])
        layer.poison()
        graph.replay()
        assert all(np.array_equal(a, b) for a, b in zip(layer.outputs(r), eager[i])), f"replay {i}"
        j = (i + 1) % 3
        other = rs[j].clone()
        layer(xs[j], other)
        assert all(np.array_equal(a, b) for a, b in zip(layer.outputs(other), eager[j]))
