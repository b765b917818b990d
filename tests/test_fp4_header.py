"""What fp4_gemm.h says of the ends of the scale range, from the formats' definitions (CPU)."""
import os
import re

import torch

from conftest import ROOT


def test_bytes_that_reach_infinity():
    with open(os.path.join(ROOT, "include", "fp4_gemm.h")) as f:
        text = " ".join(f.read().split()).replace(" * ", " ")
    named = re.search(r"bytes of (\d+) and (\d+) can reach it", text)
    largest = torch.tensor([6.0 * 2.0 ** (byte - 127) for byte in range(255)], dtype=torch.float64)
    for dtype in (torch.float32, torch.bfloat16):
        over = torch.nonzero(torch.isinf(largest.to(dtype)))[:, 0].tolist()
        assert over == [int(v) for v in named.groups()], dtype
