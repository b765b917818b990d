"""Static checks of the gfx950 assembly, kernel by kernel: every instantiation of the few-token kernels and of the FP8 x FP8
kernels whose products the compiler schedules is there, multiplies in a loop, and spills nothing (CPU only; needs hipcc)."""
import os
import re
import subprocess

import pytest

from test_kernel_asm import CSRC, HIPCC, ROOT

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")


def kernels(tmp_path, source, name):
    """{symbol: lines} of the kernels of a source whose name starts with `name`."""
    out = str(tmp_path / "out.s")
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "--cuda-device-only", "-S",
                    os.path.join(CSRC, source), "-o", out], check=True, capture_output=True)
    found = re.finditer(r"^(_ZN3moe\S*?\d+%s\S*):.*?^\.Lfunc_end" % name, open(out).read(), re.S | re.M)
    return {m.group(1): [line.strip() for line in m.group(0).splitlines()] for m in found}


def product_loops(asm):
    """Bodies of the loops that hold a product, by the compiler's notes of which loop a block is in."""
    loops, current = {}, None
    for x in asm:
        if re.match(r"(\.LBB\d+_\d+:|; %bb)", x):
            current = None
        if m := re.match(r"\.LBB(\d+_\d+):.*=>", x) or re.search(r"in Loop: Header=BB(\d+_\d+)", x):
            current = m.group(1)
        if current:
            loops.setdefault(current, []).append(x)
    return [v for v in loops.values() if any(x.startswith("v_mfma") for x in v)]


@pytest.mark.parametrize("source,name,count,loops", [
    ("few.hip", "few_linear1", 5, 6),            # the one for more than 16 tokens has a loop for experts of at most 16, too
    ("few.hip", "few_linear2", 6, 6),
    ("gemm_fp8.hip", "gemm_fp8_skinny", 8, None),
    ("gemm_fp8.hip", "gemm_fp8_tiled_f32", 1, None),
])
def test_products_in_loops_without_spills(tmp_path, source, name, count, loops):
    found = kernels(tmp_path, source, name)
    assert len(found) == count, sorted(found)
    total = 0
    for symbol, asm in found.items():
        bodies = product_loops(asm)
        assert bodies, symbol
        for body in bodies:
            assert not [x for x in body if x.startswith("scratch_")], symbol
        total += len(bodies)
    assert loops is None or total == loops
