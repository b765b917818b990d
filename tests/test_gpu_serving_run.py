"""The serving operators together, as a decoding loop uses them: bf16 activations are cast to FP8,
the gate is an FP8 GEMM with FP32 logits, the router picks the experts and moe_forward_few runs
the layer; a shared expert's down projection is another FP8 GEMM. Each step is compared with the
oracle on the previous step's own output, eagerly, on a side stream, and captured in a graph."""
import numpy as np
import pytest
import torch

from conftest import gpu_available
from gpu_helpers import Y_TOL
from test_gpu_fp8_gemm import alignment_bound
from synth import MoEConfig, make_bf16_activations, make_inputs

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

import block_scaled_fp8_dispatch_amd as moe  # noqa: E402
import oracle  # noqa: E402


class Layer:
    def __init__(self, cfg, seed=0):
        self.cfg = cfg
        inp = make_inputs(cfg, seed=seed, device="cuda")
        self.host = inp.numpy()
        self.shape = moe.make_shape(cfg.E, cfg.H, cfg.I, cfg.k, cfg.T)
        self.packed = torch.empty(moe.moe_packed_weights_bytes(self.shape), dtype=torch.uint8, device="cuda")
        moe.moe_prepare_weights(self.shape, inp.w1, inp.w1_sf, inp.w2, inp.w2_sf, self.packed)
        rng = np.random.default_rng(seed)
        sfw = 4 * -(-cfg.H // 512)
        self.gate = rng.integers(0, 0x30, (cfg.E, cfg.H)).astype(np.uint8) | (rng.integers(0, 2, (cfg.E, cfg.H)) << 7).astype(np.uint8)
        self.gate_sf = np.full((-(-cfg.E // 128), sfw), 123, dtype=np.uint8)
        self.shared = rng.integers(0, 0x70, (cfg.H, cfg.H)).astype(np.uint8)
        self.shared_sf = rng.integers(118, 122, (-(-cfg.H // 128), sfw)).astype(np.uint8)
        dev = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
        self.g_gate = (dev(self.gate), dev(self.gate_sf))
        self.g_shared = (dev(self.shared), dev(self.shared_sf))
        T, H = cfg.T, cfg.H
        self.x8 = torch.empty(T, H, dtype=torch.uint8, device="cuda")
        self.xsf = torch.empty(T, sfw, dtype=torch.uint8, device="cuda")
        self.logits = torch.empty(T, cfg.E, device="cuda")
        self.idx = torch.empty(T, cfg.k, dtype=torch.int32, device="cuda")
        self.w = torch.empty(T, cfg.k, device="cuda")
        self.y = torch.empty(T, H, dtype=torch.int16, device="cuda")
        self.z = torch.empty(T, H, dtype=torch.int16, device="cuda")
        self.ws = torch.empty(moe.moe_few_workspace_bytes(self.shape), dtype=torch.uint8, device="cuda")
        self.gws = torch.empty(moe.moe_fp8_gemm_workspace_bytes(T, 1), dtype=torch.uint8, device="cuda")

    def __call__(self, x, stream=None):
        c = self.cfg
        moe.moe_cast_to_fp8(x.view(torch.int16), c.T, c.H, self.x8, self.xsf, stream=stream)
        moe.moe_fp8_gemm(self.logits, moe.MOE_F32, self.x8, self.xsf, c.T, c.E, c.H, *self.g_gate, self.gws, stream=stream)
        moe.moe_topk_router(self.idx, self.w, self.logits, moe.MOE_F32, c.T, c.E, c.k, moe.MOE_ROUTER_SOFTMAX_CHOSEN,
                            stream=stream)
        moe.moe_forward_few(self.y, self.x8, self.xsf, self.idx, self.w, c.T, self.shape, self.packed, self.ws, stream=stream)
        moe.moe_fp8_gemm(self.z, moe.MOE_BF16, self.x8, self.xsf, c.T, c.H, c.H, *self.g_shared, self.gws, stream=stream)

    def outputs(self):
        torch.cuda.synchronize()
        return [t.cpu().numpy() for t in (self.x8, self.xsf, self.logits, self.idx, self.w, self.y, self.z)]


def _poison(layer):
    for t in (layer.x8, layer.xsf, layer.idx, layer.y, layer.z, layer.ws, layer.gws):
        t.fill_(0x7F)
    layer.logits.fill_(float("nan"))
    layer.w.fill_(float("nan"))


def test_a_decoding_step():
    cfg = MoEConfig("step", T=21, E=24, k=4, H=640, I=384)
    layer = Layer(cfg)
    xs = [make_bf16_activations(cfg.T, cfg.H, seed=s, device="cuda") for s in (1, 2, 3)]
    eager = []
    for x in xs:
        _poison(layer)
        layer(x)
        eager.append(layer.outputs())
    x8, xsf, logits, idx, w, y, z = eager[0]
    ref8, refsf = oracle.cast_to_fp8(xs[0].view(torch.int16).cpu().numpy().view(np.uint16))
    assert np.array_equal(x8, ref8) and np.array_equal(xsf, refsf)
    r = oracle.fp8_gemm(x8, xsf, layer.gate, layer.gate_sf, cfg.H)
    assert oracle.gemm_f32_within_bound(logits, r["exact"], r["bound"]).all()
    ref_idx, ref_w = oracle.topk_router(logits.astype(np.float64), cfg.k, False)
    assert np.array_equal(idx, ref_idx)
    spread = float(logits.max(1).max() - logits.min())
    assert np.abs(w - ref_w).max() <= (2 * (spread + 4) + cfg.E + 2) * 2.0 ** -24
    h = layer.host
    ref = oracle.forward(x8, xsf, idx, w, h["w1"], h["w1_sf"], h["w2"], h["w2_sf"])
    assert oracle.y_row_error(y.view(np.uint16), ref["y"]).max() <= Y_TOL
    r = oracle.fp8_gemm(x8, xsf, layer.shared, layer.shared_sf, cfg.H)
    r["bound"] = r["bound"] + alignment_bound(x8, xsf, layer.shared, layer.shared_sf, cfg.H)
    assert oracle.gemm_bf16_within_bound(z.view(np.uint16), r["exact"], r["bound"]).all()

    # on another stream than the current one
    side = torch.cuda.Stream()
    _poison(layer)
    side.wait_stream(torch.cuda.current_stream())
    layer(xs[1], stream=side)
    for got, want in zip(layer.outputs(), eager[1]):
        assert np.array_equal(got, want)

    # captured once, replayed with new activations between eager calls
    buf = xs[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(buf)
    for i in (0, 1, 2, 1, 0):
        buf.copy_(xs[i])
        _poison(layer)
        graph.replay()
        for got, want in zip(layer.outputs(), eager[i]):
            assert np.array_equal(got, want), f"replay {i}"
        layer(xs[(i + 1) % 3])
        for got, want in zip(layer.outputs(), eager[(i + 1) % 3]):
            assert np.array_equal(got, want)
