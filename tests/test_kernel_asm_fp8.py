"""Static checks of the gfx950 assembly of the tiled FP8 x FP8 GEMM and of the few-token kernels (CPU only; needs hipcc), as
test_kernel_asm.py's of the FP8 x FP4 ones: their products are inline asm too, which the compiler
neither pads for hazards nor keeps in place by itself."""
import os
import re
import subprocess

import pytest

from test_kernel_asm import CSRC, HIPCC, ROOT, _is_instr, _loops, _mfma_operands, _vregs

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{name: lines} of every instantiation of the tiled kernels."""
    out = str(tmp_path_factory.mktemp("asm") / "gemm_fp8.s")
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "--cuda-device-only", "-S",
                    os.path.join(CSRC, "gemm_fp8.hip"), "-o", out], check=True, capture_output=True)
    text = open(out).read()
    found = {m.group(1): [line.strip() for line in m.group(0).splitlines()]
             for m in re.finditer(r"^(_ZN3moe\S*gemm_fp8_(?:tiled|rounds)I\S+):.*?^\.Lfunc_end", text, re.S | re.M)}
    assert len(found) == 9
    return found


def test_no_valu_write_of_a_source_within_two_wait_states(kernels):
    for name, asm in kernels.items():
        checked = 0
        for i, line in enumerate(asm):
            if not line.startswith("v_mfma"):
                continue
            ops = _mfma_operands(line)
            src = _vregs(ops[1]) | _vregs(ops[2]) | _vregs(ops[4]) | _vregs(ops[5])
            waits, j = 0, i - 1
            while j >= 0 and waits < 2:
                p = asm[j]
                j -= 1
                if not _is_instr(p):
                    continue
                op = p.split()[0]
                if op.startswith("v_") and not op.startswith("v_mfma"):
                    dst = p.split(None, 1)[1].split(",")[0].strip()
                    assert not (_vregs(dst) & src), f"{name}: {p!r} {waits} wait states before {line!r}"
                waits += int(p.split()[1]) + 1 if op == "s_nop" else 1
            checked += 1
        assert checked >= 15 * 16, name


def test_accumulators_stay_in_place_and_nothing_spills(kernels):
    for name, asm in kernels.items():
        for line in asm:
            if line.startswith("v_mfma"):
                ops = _mfma_operands(line)
                assert ops[0] == ops[3] and ops[0].startswith("a["), f"{name}: {line}"
            assert not line.startswith("scratch_"), f"{name}: {line}"
        main = [asm[s:e] for s, e in _loops(asm) if sum(x.startswith("v_mfma") for x in asm[s:e]) >= 128]
        assert main, name
        for body in main:
            assert not [x for x in body if x.startswith("v_accvgpr")], name


def test_accumulator_reads_wait_for_the_last_product(kernels):
    for name, asm in kernels.items():
        age = {}                                 # accumulator -> wait states since its last product
        for line in asm:
            if not _is_instr(line):
                continue
            op = line.split()[0]
            if op == "v_accvgpr_read_b32":
                reg = int(re.search(r"a(\d+)", line.split(",")[1]).group(1))
                assert age.get(reg, 99) >= 19, f"{name}: {line!r} {age[reg]} wait states after its product"
            step = int(line.split()[1]) + 1 if op == "s_nop" else 1
            for r in age:
                age[r] += step
            if op.startswith("v_mfma"):
                lo, hi = map(int, re.match(r"a\[(\d+):(\d+)\]", _mfma_operands(line)[0]).groups())
                age.update({r: 0 for r in range(lo, hi + 1)})


def test_the_few_token_loops_spill_nothing(tmp_path):
    """A spilled address is loaded after the weights in flight, and waiting for it waits for them."""
    out = str(tmp_path / "few.s")
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "--cuda-device-only", "-S",
                    os.path.join(CSRC, "few.hip"), "-o", out], check=True, capture_output=True)
    asm = [line.strip() for line in open(out)]
    loops, current = {}, None                    # instructions by the loop that the compiler's notes put their block in
    for x in asm:
        if re.match(r"(\.LBB\d+_\d+:|; %bb)", x):
            current = None
        if m := re.match(r"\.LBB(\d+_\d+):.*=>This", x) or re.search(r"in Loop: Header=BB(\d+_\d+)", x):
            current = m.group(1)
        if current:
            loops.setdefault(current, []).append(x)
    products = {k: v for k, v in loops.items() if any(x.startswith("v_mfma") for x in v)}
    assert len(products) >= 9                    # five few_linear1 (one with two), three few_linear2
    for name, body in products.items():
        assert not [x for x in body if x.startswith("scratch_")], name
