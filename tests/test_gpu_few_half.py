"""The few-token forward where few_linear1 leaves half blocks of h in FP32 and few_linear2 requantises them (at most
64 slots and 32 K elements of h, H >= 1024), and at the borders of that choice. Checks and tolerances as in
test_gpu_few.py."""
import dataclasses

import numpy as np
import pytest
import torch

from conftest import gpu_available
from synth import MoEConfig, make_inputs

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

import block_scaled_fp8_dispatch_amd as moe  # noqa: E402
from test_gpu_few import FewRun, check  # noqa: E402


@pytest.mark.parametrize("cfg,max_tokens", [
    (MoEConfig("half_min", T=1, E=1, k=1, H=1024, I=128), 1),            # two blocks of 512 K for four parts of K
    (MoEConfig("half_i640", T=3, E=16, k=4, H=1536, I=640), 32),         # a last scale word of one block
    (MoEConfig("half_most", T=2, E=32, k=8, H=1152, I=2048), 2),         # 32 K elements
    (MoEConfig("half_over", T=3, E=32, k=8, H=1152, I=2048), 3),         # more: whole blocks
    (MoEConfig("half_k1", T=16, E=40, k=1, H=2176, I=512), 16),          # several x chunks per thread
    (MoEConfig("half_63", T=9, E=64, k=7, H=1280, I=256), 9),
    (MoEConfig("half_64", T=16, E=9, k=4, H=1024, I=384), 4096),
    (MoEConfig("half_66", T=11, E=9, k=6, H=1024, I=128), 11),           # more slots than lanes
    (MoEConfig("half_i128", T=8, E=70, k=8, H=1024, I=128), 8),
    (MoEConfig("wide_20", T=20, E=4, k=2, H=4352, I=256), 20),           # more than 128 workgroups of 32 columns
    (MoEConfig("narrow_20", T=20, E=4, k=2, H=4096, I=384), 32),         # 128: of 16 columns
    (MoEConfig("wide_66", T=11, E=9, k=6, H=4224, I=128), 11),
    (MoEConfig("half_shared", T=12, E=2, k=2, H=1664, I=768), 12),       # every token to both experts
], ids=lambda v: v.name if hasattr(v, "name") else str(v))
def test_parity(cfg, max_tokens):
    print(f"[few] {cfg}", flush=True)
    run = FewRun(make_inputs(cfg, seed=21, device="cuda"), max_tokens)
    y = run()
    check(run, y)
    assert np.array_equal(run(), y), "two calls gave different bytes"


def test_unused_invalid_and_repeated_ids():
    cfg = MoEConfig("half_ids", T=12, E=5, k=4, H=1024, I=256)
    inp = make_inputs(cfg, seed=5, device="cuda")
    idx = inp.topk_idx.cpu().numpy().copy()
    idx[0] = -1
    idx[1] = [7, -9, 5, 1 << 30]
    idx[2] = 3
    idx[3] = [2, -1, 2, 4]
    idx[4] = [-1, -1, -1, 0]
    run = FewRun(dataclasses.replace(inp, topk_idx=torch.from_numpy(idx).cuda()))
    y = run()
    assert (y[:2] == 0).all()
    check(run, y, idx)
    for T in (11, 5, 3, 1):
        check(run, run(T=T), idx, T)
    assert (run(topk_idx=torch.full_like(inp.topk_idx, -1)) == 0).all()


def test_nan_stays_in_its_token():
    cfg = MoEConfig("half_nan", T=8, E=6, k=2, H=1024, I=256)
    inp = make_inputs(cfg, seed=6, device="cuda")
    run = FewRun(inp)
    clean = run()
    x = inp.x_fp8.clone()
    x.view(torch.uint8)[3, 77] = 0x7F
    y = run(x_fp8=x)
    keep = [t for t in range(8) if t != 3]
    assert np.array_equal(y[keep], clean[keep])
    assert ((y[3] & 0x7FFF) > 0x7F80).all(), "the token's own outputs are not NaN"


def test_graph_replays():
    cfg = MoEConfig("half_graph", T=4, E=16, k=4, H=2048, I=512)
    inps = [make_inputs(cfg, seed=s, device="cuda") for s in (1, 2, 3)]
    run = FewRun(inps[0])
    want = [run(x_fp8=i.x_fp8, x_sf=i.x_sf, topk_idx=i.topk_idx, topk_weights=i.topk_weights) for i in inps]
    bufs = [getattr(inps[0], n).clone() for n in ("x_fp8", "x_sf", "topk_idx", "topk_weights")]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_forward_few(run.y, *bufs, cfg.T, run.shape, run.packed, run.ws[: run.nb])
    for j in (0, 1, 2, 1, 0):
        for b, n in zip(bufs, ("x_fp8", "x_sf", "topk_idx", "topk_weights")):
            b.copy_(getattr(inps[j], n))
        run.y.fill_(0)
        run.ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(run.y[: cfg.T].cpu().numpy().view(np.uint16), want[j]), j
