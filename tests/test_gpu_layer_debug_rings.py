"""The tests that go around the rings of stages and over several tiles, in the
bounds-checked debug build: a guarded access outside its buffer sets the status
that each of them looks at."""
import os
import subprocess
import sys

import pytest

from windowed_attention_implicit_b200 import build as B

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_rings_and_tiles_in_bounds():
    B.build(debug=True)
    files = [os.path.join("tests", f) for f in ("test_gpu_layer_ring.py", "test_gpu_layer_fused.py",
                                                "test_gpu_block_maps.py")]
    picked = "75001 or 30001-601 or 20003 or 606001 or 513-256 or 4000-256 or 38145 or large_map"
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "-m", "gpu", "-k", picked, *files], cwd=ROOT,
                       env={**os.environ, "RIB_DEBUG_LIBRARY": "1"}, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    assert " passed" in r.stdout
