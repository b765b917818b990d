"""GPU parity of moe_forward_few against the fp64 oracle.

The requantised intermediate is read from the workspace and compared with the oracle's: each
code must round a value within the FP32 accumulation bound of the exact h at its block's scale.
y is then compared with the oracle's Linear2 and weighted sum on the GPU's own (exactly decoded)
intermediate: |y - exact| <= bound + 2^-8 (|exact| + bound), bf16's half step, with bound =
gamma_n * sum |w h W2| for the FP32 sums in any order, n = I (products of one expert) + k (weight,
sum over experts) + 8 (the waves' partial sums) + k (the sum of a repeated expert's weights), and
end to end within 2e-2 of the row's largest value, as moe_forward.

The matrix instruction adds the products of each 8 consecutive K after aligning them to the largest
of the 8 and drops what lies more than 13 bits below its leading bit (a property of gfx950's unit for
FP8 and FP4 operands, measured with one large and one small product at every distance): each of the 8 is
off by less than 2^-13 of the group's largest product, so the bound gains 2^-10 * sum over groups of
|w| max|h| max|W2|."""
import dataclasses

import numpy as np
import pytest
import torch

from conftest import gpu_available
from gpu_helpers import Y_TOL, _HALF_GAP
from synth import MoEConfig, make_inputs

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

import block_scaled_fp8_dispatch_amd as moe  # noqa: E402
import oracle  # noqa: E402

POISON = 0x7FBF


class FewRun:
    def __init__(self, inp, max_tokens=None):
        c = inp.cfg
        self.inp, self.cfg = inp, c
        self.max_tokens = max_tokens or c.T
        self.shape = moe.make_shape(c.E, c.H, c.I, c.k, self.max_tokens)
        self.packed = torch.empty(moe.moe_packed_weights_bytes(self.shape), dtype=torch.uint8, device="cuda")
        moe.moe_prepare_weights(self.shape, inp.w1, inp.w1_sf, inp.w2, inp.w2_sf, self.packed)
        self.nb = moe.moe_few_workspace_bytes(self.shape)
        self.ws = torch.empty(self.nb + 256, dtype=torch.uint8, device="cuda")
        self.y = torch.empty(c.T + 1, c.H, dtype=torch.int16, device="cuda")

    def __call__(self, T=None, **over):
        i, T = self.inp, self.cfg.T if T is None else T
        self.ws.fill_(0xFF)
        self.y.fill_(POISON)
        v = dict(x_fp8=i.x_fp8, x_sf=i.x_sf, topk_idx=i.topk_idx, topk_weights=i.topk_weights)
        v.update(over)
        moe.moe_forward_few(self.y, v["x_fp8"], v["x_sf"], v["topk_idx"], v["topk_weights"], T, self.shape, self.packed,
                            self.ws[: self.nb])
        torch.cuda.synchronize()
        assert (self.ws[self.nb:] == 0xFF).all(), "a store went past the workspace"
        y = self.y.cpu().numpy().view(np.uint16)
        assert (y[T:] == POISON).all(), "a store went past the last token"
        return y[:T].copy()

    def intermediate(self):
        """codes [S, I] and scale bytes [S, I/128] as the workspace holds them."""
        c = self.cfg
        S = min(self.max_tokens, moe.MOE_FEW_MAX_TOKENS) * c.k
        raw = self.ws[: self.nb].cpu().numpy()
        o = -(-S * c.I // 256) * 256
        sfs = 4 * -(-c.I // 512)
        return raw[: S * c.I].reshape(S, c.I), raw[o: o + S * sfs].reshape(S, sfs)[:, : c.I // 128]


def check(run, y, idx=None, T=None):
    inp, c = run.inp.numpy(), run.cfg
    T = c.T if T is None else T
    idx = inp["topk_idx"] if idx is None else idx
    idx, w = idx[:T], inp["topk_weights"][:T].astype(np.float64)
    args = (inp["x_fp8"][:T], inp["x_sf"][:T], idx, inp["topk_weights"][:T], inp["w1"], inp["w1_sf"], inp["w2"], inp["w2_sf"])
    ref = oracle.forward(*args, keep_bounds=True)
    codes, sf = run.intermediate()
    hd = {}
    for t in range(T):
        for j in range(c.k):
            e = int(idx[t, j])
            if not 0 <= e < c.E:
                continue
            s, first = t * c.k + j, t * c.k + int(np.nonzero(idx[t] == e)[0][0])
            q, b = codes[first], np.repeat(sf[first], 128)
            assert (b != 255).all() and not np.isnan(oracle.E4M3_TABLE[q]).any()
            scale = np.ldexp(1.0, b.astype(np.int64) - 127)
            hd[s] = oracle.E4M3_TABLE[q] * scale
            off = np.abs(hd[s] - ref["h"][s]) - ref["h_bound"][s] - _HALF_GAP[q] * scale
            assert (off <= 0).all(), f"token {t} expert {e}: intermediate column {off.argmax()}"
    out = oracle.linear2_combine(hd, idx, inp["topk_weights"][:T], inp["w2"], inp["w2_sf"])["y"]
    mag, aligned = np.zeros_like(out), np.zeros_like(out)
    for e in range(c.E):
        sl = [(t, j) for t in range(T) for j in range(c.k) if int(idx[t, j]) == e]
        if sl:
            W = np.abs(oracle.dequant_fp4_rows(inp["w2"][e], inp["w2_sf"][e], c.I))
            W8 = W.reshape(c.H, c.I // 8, 8).max(2)
            for t, j in sl:
                h = np.abs(hd[t * c.k + j])
                mag[t] += abs(w[t, j]) * (W @ h)
                aligned[t] += 2.0 ** -10 * abs(w[t, j]) * (W8 @ h.reshape(c.I // 8, 8).max(1))
    n = c.I + 2 * c.k + 8
    bound = n * 2.0 ** -24 / (1 - n * 2.0 ** -24) * mag + aligned
    assert oracle.gemm_bf16_within_bound(y, out, bound).all()
    err = oracle.y_row_error(y, ref["y"])
    print(f"[few] {c} T={T}: max row error {err.max():.3e}", flush=True)
    assert err.max() <= Y_TOL


@pytest.mark.parametrize("cfg,max_tokens", [
    (MoEConfig("few_min", T=1, E=1, k=1, H=128, I=128), 1),
    (MoEConfig("few_c0", T=3, E=4, k=2, H=256, I=512), 8),
    (MoEConfig("few_odd16", T=16, E=8, k=2, H=384, I=640), 16),
    (MoEConfig("few_17", T=17, E=8, k=3, H=640, I=384), 20),
    (MoEConfig("few_32", T=32, E=32, k=8, H=1024, I=256), 4096),
    (MoEConfig("few_deep", T=5, E=2, k=2, H=512, I=1152), 5),
    (MoEConfig("few_e70", T=7, E=70, k=6, H=256, I=128), 7),
    (MoEConfig("few_k64", T=32, E=64, k=64, H=128, I=128), 32),
    (MoEConfig("few_e1024", T=9, E=1024, k=4, H=128, I=128), 9),
    (MoEConfig("few_one", T=1, E=4, k=2, H=7168, I=2048), 1),
    (MoEConfig("few_x_lds", T=16, E=3, k=2, H=7168, I=256), 16),         # x in LDS at its largest
    (MoEConfig("few_x_big", T=16, E=3, k=2, H=7936, I=128), 16),         # x too large for LDS
    (MoEConfig("few_h1920", T=29, E=6, k=4, H=1920, I=896), 31),
], ids=lambda v: v.name if hasattr(v, "name") else str(v))
def test_few_parity(cfg, max_tokens):
    print(f"[few] {cfg}", flush=True)
    run = FewRun(make_inputs(cfg, seed=11, device="cuda"), max_tokens)
    y = run()
    check(run, y)
    assert np.array_equal(run(), y), "two calls gave different bytes"


def test_few_unused_invalid_and_repeated_ids():
    cfg = MoEConfig("few_ids", T=19, E=5, k=4, H=256, I=256)
    inp = make_inputs(cfg, seed=3, device="cuda")
    idx = inp.topk_idx.cpu().numpy().copy()
    idx[0] = -1                          # no slot at all
    idx[1] = [7, -9, 5, 1 << 30]         # nothing valid
    idx[2] = 3                           # the same expert four times
    idx[3] = [2, -1, 2, 4]
    idx[4] = [-1, -1, -1, 0]
    run = FewRun(dataclasses.replace(inp, topk_idx=torch.from_numpy(idx).cuda()))
    y = run()
    assert (y[:2] == 0).all(), "a token without a valid slot is not zero"
    check(run, y, idx)
    # fewer tokens than the tensors hold, down to one; none at all
    for T in (18, 16, 5, 1):
        yt = run(T=T)
        check(run, yt, idx, T)
    assert run(T=0).shape[0] == 0
    # every slot unused
    y = run(topk_idx=torch.full_like(inp.topk_idx, -1))
    assert (y == 0).all()


def test_few_nan_stays_in_its_token():
    cfg = MoEConfig("few_nan", T=20, E=6, k=2, H=384, I=256)
    run = FewRun(make_inputs(cfg, seed=4, device="cuda"))
    clean = run()
    x = run.inp.x_fp8.clone()
    x[7, 130] = 0x7F
    x_sf = run.inp.x_sf.clone()
    x_sf[18, 1] = 255
    y = run(x_fp8=x, x_sf=x_sf)
    vals = oracle.bf16_bits_to_f64(y)
    assert np.isnan(vals[[7, 18]]).all()
    keep = [t for t in range(20) if t not in (7, 18)]
    assert np.array_equal(y[keep], clean[keep])
    # a NaN weight scale of an expert reaches the tokens that chose it, no others
    idx = run.inp.topk_idx.cpu().numpy()
    e = int(idx[0, 0])
    w2_sf = run.inp.w2_sf.clone()
    w2_sf[e, 5, 1] = 255
    bad = FewRun(dataclasses.replace(run.inp, w2_sf=w2_sf))
    y = bad()
    hit = (idx == e).any(1)
    vals = oracle.bf16_bits_to_f64(y)
    assert np.isnan(vals[hit, 5]).all()
    vals[:, 5] = 0
    assert np.isfinite(vals).all()
    assert np.array_equal(y[~hit], clean[~hit])


def test_few_on_a_forward_workspace_and_near_the_forward():
    cfg = MoEConfig("few_vs", T=32, E=16, k=4, H=512, I=512)
    inp = make_inputs(cfg, seed=6, device="cuda")
    run = FewRun(inp, max_tokens=200)
    y = run()
    ws = torch.empty(moe.moe_workspace_bytes(run.shape), dtype=torch.uint8, device="cuda")
    y2 = torch.empty(32, cfg.H, dtype=torch.int16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_forward_few(y2, inp.x_fp8, inp.x_sf, inp.topk_idx, inp.topk_weights, 32, run.shape, run.packed, ws, stream=side)
    torch.cuda.synchronize()
    assert np.array_equal(y2.cpu().numpy().view(np.uint16), y)
    moe.moe_forward(y2, inp.x_fp8, inp.x_sf, inp.topk_idx, inp.topk_weights, 32, run.shape, run.packed, ws)
    torch.cuda.synchronize()
    err = oracle.y_row_error(y, oracle.bf16_bits_to_f64(y2.cpu().numpy().view(np.uint16)))
    assert err.max() <= Y_TOL


def test_few_graph_replays_match_eager():
    cfg = MoEConfig("few_graph", T=12, E=8, k=2, H=512, I=384)
    trials = [make_inputs(cfg, seed=s, device="cuda") for s in (1, 2, 3)]
    base = trials[0]
    names = ("x_fp8", "x_sf", "topk_idx", "topk_weights")
    run = FewRun(base)
    eager = [run(**{n: getattr(t, n) for n in names}) for t in trials]
    assert not np.array_equal(eager[0], eager[1])
    buf = {n: getattr(base, n).clone() for n in names}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_forward_few(run.y, buf["x_fp8"], buf["x_sf"], buf["topk_idx"], buf["topk_weights"], cfg.T, run.shape,
                            run.packed, run.ws)
    for i in (0, 1, 2, 1, 0):
        for n in names:
            buf[n].copy_(getattr(trials[i], n))
        run.y.fill_(POISON)
        run.ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(run.y[: cfg.T].cpu().numpy().view(np.uint16), eager[i]), f"replay {i}"
