"""GPU parity of the norm with FP8 output at many rows, where a thread holds two to four chunks of a row, and at the borders of
those choices. Rows at both ends and in between are checked against the oracle (as test_gpu_rmsnorm.py's), all of them against
each other: the rows repeat, so that every copy of one has to give the same bytes."""
import numpy as np
import pytest
import torch

from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

import block_scaled_fp8_dispatch_amd as moe  # noqa: E402
from test_gpu_rmsnorm import bf16, call, check, rows  # noqa: E402

DIFFERENT = 16


@pytest.mark.parametrize("wf32,residual", [(False, True), (True, False)])
@pytest.mark.parametrize("R", [1023, 1024, 1041])
@pytest.mark.parametrize("C", [128, 2048, 2176, 4096, 4224, 8192, 8320, 16384, 16512, 24576, 24704, 32768, 32896])
def test_many_rows(R, C, wf32, residual):
    print(f"[norm] {R} {C} {residual} {wf32}", flush=True)
    index = torch.arange(R, device="cuda") % DIFFERENT
    x = rows(DIFFERENT, C, C)[index]
    res = rows(DIFFERENT, C, C + 1, 3.0)[index] if residual else None
    w = 1 + 0.2 * torch.randn(C, generator=torch.Generator(device="cuda").manual_seed(C), device="cuda")
    w = w if wf32 else bf16(w)
    got = call(x, res, w, 1e-6)
    for v in got:
        whole = v[: R // DIFFERENT * DIFFERENT].reshape(-1, DIFFERENT, v.shape[1])
        assert (whole == whole[0]).all() and np.array_equal(v[len(whole) * DIFFERENT:], v[: R % DIFFERENT])
    check([v[:DIFFERENT] for v in got], x[:DIFFERENT], None if res is None else res[:DIFFERENT], w, 1e-6)


def test_two_streams_at_once():
    """Nothing is shared between calls: two on streams of their own, many times over."""
    cases = []
    for C, R in ((7168, 2000), (18432, 1500)):
        x, res = rows(R, C, C), rows(R, C, C + 1)
        w = bf16(torch.ones(C, device="cuda") * 1.5)
        sf = 4 * -(-C // 512)
        out = [torch.empty(R, C, dtype=torch.uint8, device="cuda"), torch.empty(R, sf, dtype=torch.uint8, device="cuda"),
               torch.empty(R, C, dtype=torch.bfloat16, device="cuda"), torch.empty(R, C, dtype=torch.bfloat16, device="cuda")]
        cases.append((torch.cuda.Stream(), x, res, w, out, call(x, res, w, 1e-5)))
    for _ in range(6):
        for stream, x, res, w, out, _ in cases:
            moe.moe_rmsnorm_to_fp8(*out, x, res, w, moe.MOE_BF16, x.shape[0], x.shape[1], 1e-5, stream=stream.cuda_stream)
    torch.cuda.synchronize()
    for *_, out, want in cases:
        for a, b in zip(out, want):
            assert np.array_equal(a.cpu().view(torch.uint8 if a.dtype == torch.uint8 else torch.int16).numpy().view(b.dtype), b)


def test_captured_and_replayed():
    """The row count and the pointers are the graph's; contents may change between replays."""
    R, C = 1200, 4224
    x, res = rows(R, C, 1), rows(R, C, 2)
    w = torch.linspace(0.5, 1.5, C, device="cuda")
    q = torch.empty(R, C, dtype=torch.uint8, device="cuda")
    sf = torch.empty(R, 4 * -(-C // 512), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        moe.moe_rmsnorm_to_fp8(q, sf, None, out, x, res, w, moe.MOE_F32, R, C, 1e-5, stream=torch.cuda.current_stream().cuda_stream)
    for seed in range(3):
        x.copy_(rows(R, C, 10 + seed))
        graph.replay()
        torch.cuda.synchronize()
        want = call(x, res, w, 1e-5, normed=False)
        assert np.array_equal(q.cpu().numpy(), want[0]) and np.array_equal(sf.cpu().numpy(), want[1])
        assert np.array_equal(out.cpu().view(torch.int16).numpy().view(np.uint16), want[3])
