"""The C library stands without torch: building it, finding it built, loading
it and calling it on raw pointers."""
import os
import subprocess
import sys

import linear_fp16_gb300 as L
from linear_fp16_gb300 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIDE = "import sys; sys.modules['torch'] = None\n"   # import torch raises ImportError


def _python(code):
    r = subprocess.run([sys.executable, "-c", HIDE + code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


def test_the_library_loads_and_answers_without_torch():
    L.load_library()  # built
    out = _python("import linear_fp16_gb300 as L\n"
                  "from linear_fp16_gb300 import build as B, ffn\n"
                  "assert B.up_to_date() and L.poot_linear_version() > 0\n"
                  "assert L.poot_gated_linear(None, 0) == L.POOT_ERR_INVALID_ARG\n"
                  "assert ffn.load_library() is L.load_library()\n"
                  "print('loaded')")
    assert out == "loaded\n"


def test_the_library_is_built_without_torch(tmp_path):
    """With the compiler replaced: the commands are nvcc's, on CUDA sources only."""
    out = _python("from linear_fp16_gb300 import build as B\n"
                  f"B.BUILD = {str(tmp_path)!r}; B.LIB = B.os.path.join(B.BUILD, 'lib.so')\n"
                  "cmds = []\n"
                  "def run(cmd, verbose):\n"
                  "    cmds.append(cmd)\n"
                  "    open(cmd[cmd.index('-o') + 1], 'w').close()\n"
                  "B._run = run\n"
                  "assert not B.up_to_date()\n"
                  "assert B.build() == B.LIB and B.up_to_date()\n"
                  "assert len(cmds) == len(B.SOURCES) + 1 and all('nvcc' in c[0] for c in cmds)\n"
                  "assert not any('torch' in a for c in cmds for a in c)\n"
                  "print('built')")
    assert out == "built\n" and os.listdir(tmp_path) == ["lib.so"]


def test_another_torch_rebuilds_the_extension_alone(tmp_path, monkeypatch):
    cmds = []

    def run(cmd, verbose):
        cmds.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
    B.build()
    monkeypatch.setattr(B, "_run", run)
    monkeypatch.setattr(B, "extension", lambda: str(tmp_path / "ext.so"))
    assert B.up_to_date() and not B.extension_up_to_date()
    assert B.build_extension() == str(tmp_path / "ext.so") and B.extension_up_to_date()
    assert [c[0] for c in cmds] == ["g++", "g++"]
