"""Checks on the gfx950 assembly of the norm, the 4-bit products and the page calls (CPU only): nothing in scratch memory,
no packed 32-bit arithmetic, and the products' loops keep the next steps' loads in flight."""
import os
import re
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

from bit_quantized_moe_02_amd import build as B  # noqa: E402

HIPCC = B.HIPCC if shutil.which(B.HIPCC) or os.path.exists(B.HIPCC) else None
pytestmark = pytest.mark.skipif(HIPCC is None, reason="hipcc not available")


def assembly(src, tmp_path):
    out = str(tmp_path / "k.s")
    subprocess.run([HIPCC] + B.HIP_FLAGS + ["-S", "--cuda-device-only", "-o", out, os.path.join(B.CSRC, src)], check=True, capture_output=True)
    with open(out) as f:
        return f.read()


# Norm: 3 types of x, 4 of the residual, 8 widths.  Products: 3 sizes of groups, zero points or not (and, for 8-bit rows, scales
# of a row or of groups), 9 splits over workgroups.  Pages: 2 sizes of pools for 3 decisions, giving back, 2 copies.
@pytest.mark.parametrize("src,kernels", [("k_norm.hip", 96), ("k_linear_bf16.hip", 54), ("k_linear_f16.hip", 54), ("k_linear_i8.hip", 108), ("k_pages.hip", 9)])
def test_nothing_in_scratch(src, kernels, tmp_path):
    text = assembly(src, tmp_path)
    assert not re.search(r"^\s*(scratch|flat)_", text, re.M)
    assert not re.search(r"^\s*v_pk_(add|mul|fma)_f32", text, re.M)
    seen = re.findall(r"\.name:\s+(_Z\w+)\n(.*?)\.wavefront_size", text, re.S)
    assert len(seen) == kernels
    for name, meta in seen:
        value = lambda key: int(re.search(rf"\.{key}:\s+(\d+)", meta).group(1))  # noqa: E731
        assert value("vgpr_spill_count") == 0, name
        assert value("private_segment_fixed_size") == 0, name
    for m in re.finditer(r"^(_Z\w*linear_kernelILi(\d)ELi\d+ELi(\d+)ELi(\d)E\w*):.*?\n(.*?)^\.Lfunc_end", text, re.M | re.S):
        name, body, rows, tiles = m.group(1), m.group(5), min(int(m.group(3)), 32), int(m.group(4))
        x = max(1, rows * (8 if m.group(2) == "3" else 16) // 64)               # loads of a step's rows, and of the codes of its weights
        waits = [int(c) for c in re.findall(r"vmcnt\((\d+)\)", body)]
        assert max(waits) >= x + tiles, (name, sorted(set(waits)))
