"""Checks on the gfx950 assembly of the attention kernels (CPU only), for every size of head: no vector register and no
operand lies in scratch memory.  Scalar registers may be kept in lanes of a vector register, and the prompt kernels
reserve (and never touch) 68 bytes a thread for that."""
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


@pytest.mark.parametrize("src,kernels", [("k_kv.hip", 12), ("k_attn_decode.hip", 34), ("k_attn_prefill.hip", 12)])
def test_nothing_in_scratch(src, kernels, tmp_path):
    out = str(tmp_path / "k.s")
    subprocess.run([HIPCC] + B.HIP_FLAGS + ["-S", "--cuda-device-only", "-o", out, os.path.join(B.CSRC, src)], check=True, capture_output=True)
    with open(out) as f:
        text = f.read()
    assert not re.search(r"^\s*(scratch|flat)_", text, re.M)
    seen = re.findall(r"\.name:\s+(_Z\w+)\n(.*?)\.wavefront_size", text, re.S)
    assert len(seen) == kernels
    for name, meta in seen:
        value = lambda key: int(re.search(rf"\.{key}:\s+(\d+)", meta).group(1))  # noqa: E731
        assert value("vgpr_spill_count") == 0, name
        assert value("private_segment_fixed_size") <= (68 if "prefill_kernel" in name else 0), name
