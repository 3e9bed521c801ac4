"""Checks on the gfx950 assembly of the attention kernels (CPU only) that no
numerical test can see.

* No registers in scratch memory, up to heads of 128: what rare branches need
  is computed there and not carried through the loops, and the prompt
  kernel's operands are in registers.
* The decode kernels for long contexts keep the next step's loads in flight:
  some wait leaves at least a block's worth of loads outstanding.
* The prompt kernel waits for its copies into LDS only in front of a barrier.
  A copy is behind a whole tile of work there; the compiler would wait for it
  at once where it does not know which LDS buffer a read is from.
"""
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


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{mangled name: assembly} of the attention kernels."""
    d, got = str(tmp_path_factory.mktemp("asm")), {}
    for src in ("k_kv.hip", "k_attn_decode.hip", "k_attn_prefill.hip"):
        out = os.path.join(d, src + ".s")
        subprocess.run([HIPCC] + B.HIP_FLAGS + ["-S", "--cuda-device-only", "-o", out, os.path.join(B.CSRC, src)], check=True,
                       capture_output=True)
        with open(out) as f:
            text = f.read()
        for m in re.finditer(r"^(_Z\w+):.*?\n(.*?)^\.Lfunc_end", text, re.M | re.S):
            got[m.group(1)] = m.group(2)
    return got


def test_no_scratch(kernels):
    names = [n for n in kernels if "ELi64E" in n or "ELi128E" in n]
    assert len(names) >= 2 * (2 + 2 + 5 + 1 + 4), names
    for n in names:
        assert not re.search(r"^\s*scratch_", kernels[n], re.M), n


def test_decode_keeps_loads_in_flight(kernels):
    for n, body in kernels.items():
        if "decode_kernel" in n and "ELb0E" in n:      # (the kernels for long contexts)
            loads = 2 * (2 if "ELi128E" in n else 1 if "ELi64E" in n else 4)   # of a step's K or V codes
            counts = [int(c) for c in re.findall(r"vmcnt\((\d+)\)", body)]
            assert max(counts) >= loads, (n, sorted(set(counts)))


def test_prompt_kernel_waits_for_copies_at_barriers_only(kernels):
    for n, body in kernels.items():
        if "prefill_kernel" not in n or "ELi256E" in n:
            continue
        lines = [l.strip() for l in body.splitlines() if l.strip() and not l.strip().startswith(";")]
        copies = [i for i, l in enumerate(lines) if re.match(r"buffer_load_dwordx4.*lds", l)]
        assert len(copies) > 8, n
        for i in copies:
            # what comes first behind a copy: a barrier (its wait right in front of it), not a wait among the reads
            for j in range(i + 1, len(lines)):
                if lines[j].startswith("s_barrier"):
                    break
                if "vmcnt(0)" in lines[j]:
                    assert any(x.startswith("s_barrier") for x in lines[j:j + 8]), (n, lines[j - 2:j + 4])
                    break
                if lines[j].startswith(".LBB") and j - i > 40:
                    break                    # (past the block that the copy is in)
