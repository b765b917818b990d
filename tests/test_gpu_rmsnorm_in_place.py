"""The norm with FP8 output where residual_out is the residual, or x, at sizes of every form that the launch chooses from: one to four
chunks of a row a thread, kept in the caches and not, and rows that the threads take in turn. All outputs are those of a call
with buffers of their own, byte for byte."""
import pytest
import torch

from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

import block_scaled_fp8_dispatch_amd as moe  # noqa: E402


@pytest.mark.parametrize("wf32", [False, True])
@pytest.mark.parametrize("which", ["x", "residual"])
@pytest.mark.parametrize("rows,cols", [(17, 2048), (200, 7168), (60, 10240), (120, 10240), (1200, 7168), (1200, 10240), (30, 16512), (600, 16384), (520, 24576),
                                       (300, 32768), (3, 33024), (40, 49152)])
def test_in_place(rows, cols, which, wf32):
    print(f"[norm] {rows} x {cols} {which} {wf32}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    x, res = (torch.randn(rows, cols, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = torch.rand(cols, generator=g, device="cuda") + 0.5
    w = w if wf32 else w.to(torch.bfloat16)
    ty = moe.MOE_F32 if wf32 else moe.MOE_BF16

    def call(x, res, out):
        q = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
        sf = torch.empty(rows, 4 * -(-cols // 512), dtype=torch.uint8, device="cuda")
        normed = torch.empty_like(x)
        moe.moe_rmsnorm_to_fp8(q, sf, normed, out, x, res, w, ty, rows, cols, 1e-5)
        torch.cuda.synchronize()
        return q, sf, normed.view(torch.int16), out.view(torch.int16)

    want = call(x, res, torch.empty_like(x))
    assert torch.equal(want[3].view(torch.bfloat16), (x.float() + res.float()).to(torch.bfloat16))
    a, b = x.clone(), res.clone()
    got = call(a, b, a if which == "x" else b)
    assert all(torch.equal(v, u) for v, u in zip(got, want))
    kept, was = (b, res) if which == "x" else (a, x)
    assert torch.equal(kept, was)
