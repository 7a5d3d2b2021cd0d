"""The LM head's operators give the same bits launched with programmatic dependent launch (the
default) and plainly (LORA_PDL=0), and in the checked build, whose TMA producers test every tile's
origin and which has to report nothing.  Each setting runs in its own subprocess."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "qlora_linear_b200")


def _run(**env):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "head_worker.py")], cwd=ROOT,
                       env=dict(os.environ, **env), capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    d = json.loads([ln for ln in r.stdout.splitlines() if ln.startswith("{")][-1])
    assert d["status"] and not any(d["status"])
    return d


def test_same_bits_plainly_launched_and_in_the_checked_build():
    sys.path.insert(0, PKG)
    import build
    base = _run(LORA_PDL="1")
    assert len(base["cases"]) == 5
    assert _run(LORA_PDL="0")["cases"] == base["cases"]
    checked = _run(LORA_LIB_PATH=build.build(checked=True))
    assert checked["lib"] == "liblora_linear_checked.so" and checked["cases"] == base["cases"]
