"""Static check of the gfx950 assembly of the norm with FP8 output (CPU only; needs hipcc): its forms differ."""
import os
import re
import subprocess

import pytest

from test_kernel_asm import CSRC, HIPCC, ROOT

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")


def test_no_two_forms_are_the_same_code(tmp_path):
    """One to four chunks a thread, by the weights' type and whether past the caches; rows taken in turn, by the weights' type."""
    out = str(tmp_path / "norm.s")
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "--cuda-device-only", "-S",
                    os.path.join(CSRC, "norm.hip"), "-o", out], check=True, capture_output=True)
    text = open(out).read()
    forms = {}
    for m in re.finditer(r"^(_ZN3moe\S*rmsnorm_kernel\S+):.*?^\.Lfunc_end", text, re.S | re.M):
        code = [line.split(";")[0].strip() for line in m.group(0).splitlines()[1:]]
        code = tuple(re.sub(r"\.LBB\d+_", ".LBB_", c) for c in code if re.match(r"[vsgdb]\w*_", c))
        assert len(code) > 100, m.group(1)
        forms[m.group(1)] = code
    assert len(forms) == 4 * 2 * 2 + 2
    assert len(set(forms.values())) == len(forms)
