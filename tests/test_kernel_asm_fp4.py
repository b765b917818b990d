"""Static checks of the gfx950 assembly of the FP4 x FP4 GEMMs (CPU only; needs hipcc), as test_kernel_asm.py's of the
FP8 x FP4 ones: the tiled kernels' products are inline asm, which the compiler neither pads for hazards nor keeps in place by
itself. The kernels whose waves share K multiply in a loop and spill nothing."""
import os
import re
import subprocess

import pytest

from test_kernel_asm import CSRC, HIPCC, ROOT, _is_instr, _loops, _mfma_operands, _vregs
from test_kernel_asm_spills import product_loops

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")


@pytest.fixture(scope="module")
def text(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("asm") / "gemm_fp4.s")
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "--cuda-device-only", "-S",
                    os.path.join(CSRC, "gemm_fp4.hip"), "-o", out], check=True, capture_output=True)
    return open(out).read()


def bodies(text, name):
    return {m.group(1): [line.strip() for line in m.group(0).splitlines()]
            for m in re.finditer(r"^(_ZN3moe\S*%sI\S+):.*?^\.Lfunc_end" % name, text, re.S | re.M)}


@pytest.fixture(scope="module")
def tiled(text):
    """{name: lines}: 128 rows, 64 rows with four blocks of scales a load and with one, each by output type and B's loads; and
    the 256-row tiles with their last round's parts, by output type."""
    found = bodies(text, "gemm_fp4_tiled") | bodies(text, "gemm_fp4_rounds")
    assert len(found) == 14
    return found


def written(line):
    """VGPRs that a VALU instruction writes: its first operand, and of a swap its second too."""
    op, rest = line.split(None, 1)
    operands = [o.strip() for o in rest.split(",")]
    return _vregs(operands[0]) | (_vregs(operands[1].split()[0]) if "swap" in op else set())


def test_no_valu_write_of_a_source_within_two_wait_states(tiled):
    for name, asm in tiled.items():
        checked = 0
        for i, line in enumerate(asm):
            if not line.startswith("v_mfma"):
                continue
            ops = _mfma_operands(line)
            src = _vregs(ops[1]) | _vregs(ops[2]) | _vregs(ops[4]) | _vregs(ops[5])
            assert len(_vregs(ops[1])) == len(_vregs(ops[2])) == 4 and len(_vregs(ops[4]) | _vregs(ops[5])) == 2
            waits, j = 0, i - 1
            while j >= 0 and waits < 2:
                p = asm[j]
                j -= 1
                if not _is_instr(p):
                    continue
                op = p.split()[0]
                if op.startswith("v_") and not op.startswith("v_mfma"):
                    assert not (written(p) & src), f"{name}: {p!r} {waits} wait states before {line!r}"
                waits += int(p.split()[1]) + 1 if op == "s_nop" else 1
            checked += 1
        assert checked >= 7 * 2 * 16, name                 # seven steps of two halves, at least 4 x 4 products each


def test_accumulators_stay_in_place_and_the_loops_spill_nothing(tiled):
    for name, asm in tiled.items():
        for line in asm:
            if line.startswith("v_mfma"):
                ops = _mfma_operands(line)
                assert ops[0] == ops[3] and ops[0].startswith("a["), f"{name}: {line}"
        main = [asm[s:e] for s, e in _loops(asm) if sum(x.startswith("v_mfma") for x in asm[s:e]) >= 128]
        assert len(main) == (3 if "rounds" in name else 1), name
        for body in main:
            assert not [x for x in body if x.startswith(("v_accvgpr", "scratch_"))], name


def test_accumulator_reads_wait_for_the_last_product(tiled):
    for name, asm in tiled.items():
        age, read = {}, 0                        # accumulator -> wait states since its last product
        for line in asm:
            if not _is_instr(line):
                continue
            op = line.split()[0]
            if op == "v_accvgpr_read_b32" or "_store_" in op:      # (FP32 outputs are stored from the accumulators)
                for m in re.finditer(r"\ba(?:(\d+)\b|\[(\d+):(\d+)\])", line.split(None, 1)[1]):
                    lo, hi = (int(m.group(1)),) * 2 if m.group(1) else (int(m.group(2)), int(m.group(3)))
                    for reg in range(lo, hi + 1):
                        assert age.get(reg, 99) >= 19, f"{name}: {line!r} {age[reg]} wait states after its product"
                        read += 1
            step = int(line.split()[1]) + 1 if op == "s_nop" else 1
            for r in age:
                age[r] += step
            if op.startswith("v_mfma"):
                lo, hi = map(int, re.match(r"a\[(\d+):(\d+)\]", _mfma_operands(line)[0]).groups())
                age.update({r: 0 for r in range(lo, hi + 1)})
        assert read >= 64, name


def test_every_counted_load_is_there(tiled):
    """64-row tiles: at a step's second barrier the loads behind its first may be in flight, and their number is a constant of
    the wait. Were one of them left out (the compiler drops loads whose result nothing uses), the wait would let older ones, the
    next step's rows of A, be in flight too. A step that the wait for all loads follows is the last."""
    for name, asm in tiled.items():
        if "ILi64E" not in name:
            continue
        barriers, loads, waited = [], 0, None
        for line in asm:
            if line.startswith("buffer_load"):
                loads += 1
            elif line.startswith("s_barrier"):
                barriers.append((waited, loads))
                loads = 0
            elif m := re.match(r"s_waitcnt vmcnt\((\d+)\)( lgkmcnt\(0\))?$", line):
                waited = (int(m.group(1)), bool(m.group(2)))
            elif _is_instr(line):
                waited = None
        steps = 0
        for (wait, issued), (after, _) in zip(barriers, barriers[1:] + [(None, 0)]):
            if wait and wait[1]:                             # a step's second barrier
                steps += 1
                assert issued >= wait[0] or after == (0, False), f"{name}: {issued} loads, {wait[0]} counted"
        assert steps == 7, name


def test_the_kernels_whose_waves_share_k(text):
    found = bodies(text, "gemm_fp4_skinny")
    assert len(found) == 5 * 4                             # tile shapes; output types, B's loads
    for name, asm in found.items():
        loops = product_loops(asm)
        assert loops, name
        assert not [x for x in asm if x.startswith("scratch_")], name


def test_the_cast_uses_the_conversion_instructions(tmp_path):
    """Both ways, and no scratch memory."""
    for source, wanted in (("cast_fp4.hip", ("v_cvt_scalef32_pk_fp4_f32", "v_cvt_scalef32_pk_f32_fp4", "v_cvt_scalef32_pk_bf16_fp4")),
                           ("norm.hip", ())):
        out = str(tmp_path / "out.s")
        subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "--cuda-device-only", "-S",
                        os.path.join(CSRC, source), "-o", out], check=True, capture_output=True)
        asm = [line.strip() for line in open(out)]
        for op in wanted:
            assert any(x.startswith(op) for x in asm), op
        assert not [x for x in asm if x.startswith("scratch_")], source
