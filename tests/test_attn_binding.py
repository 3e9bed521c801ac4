"""CPU checks of what the Python binding needs: the expert layer's calls work where the attention calls' module is
missing or torch lacks a short way, and the build goes on without that module."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

LAYER_CALLS = """
assert qmoe.moe_codebook_generate(1).shape == (256, 8)
assert qmoe.moe_kv_code_bytes(1, 16, 1, 64) == 2 * 16 * 64 and len(qmoe.moe_rope_freqs(64)) == 32
"""


def _python(code):
    return subprocess.run([sys.executable, "-c", "import sys\nsys.path.insert(0, %r)\nimport torch\n" % ROOT + code], cwd=ROOT,
                          stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=300)


def test_layer_calls_without_the_attention_module():
    r = _python("""
sys.modules["bit_quantized_moe_02_amd._attn"] = None
from bit_quantized_moe_02_amd import qmoe
""" + LAYER_CALLS + """
import types
qmoe._device = lambda: 0
step = types.SimpleNamespace(device=0, kv_heads=1, head_dim=64, rows=1, at=0)
x = types.SimpleNamespace(is_cuda=True)
for call in (lambda: qmoe.moe_kv_append(step, step, x, x, stream=0), lambda: qmoe.moe_kv_read(step, step, x, x, stream=0),
             lambda: qmoe.moe_attn_decode(step, step, x, x, x, 0.1, stream=0),
             lambda: qmoe.moe_attn_prefill(x, x, x, x, x, 1, x, x, 0.1, stream=0)):
    try:
        call()
    except ImportError as e:
        assert "_attn.so" in str(e)
    else:
        raise AssertionError("no error")
print("fine")
""")
    assert r.returncode == 0 and r.stdout.endswith("fine\n"), r.stdout


def test_import_without_torchs_short_ways():
    r = _python("""
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
from bit_quantized_moe_02_amd import qmoe
""" + LAYER_CALLS + "assert qmoe._device is torch.cuda.current_device\nprint('fine')\n")
    assert r.returncode == 0 and r.stdout.endswith("fine\n"), r.stdout


@pytest.mark.parametrize("error", [RuntimeError("Python.h: No such file"), OSError("no compiler"), AttributeError("no torch")])
def test_build_goes_on_without_the_attention_module(monkeypatch, tmp_path, capsys, error):
    sys.path.insert(0, ROOT)
    from bit_quantized_moe_02_amd import build as B

    def run(cmd):
        open(cmd[cmd.index("-o") + 1], "w").close()
        return ""

    def fails():
        raise error

    stale = tmp_path / "_attn.so"
    stale.write_text("of another torch")
    for name, value in (("_run", run), ("build_py_attn", fails), ("BUILD", str(tmp_path / "b")), ("LIB", str(tmp_path / "lib.so")),
                        ("PY_ATTN", str(stale))):
        monkeypatch.setattr(B, name, value)
    assert B.build() == str(tmp_path / "lib.so") and os.path.exists(tmp_path / "lib.so")
    assert not stale.exists() and str(error) in capsys.readouterr().err
