"""The serving example runs and its own comparisons hold."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_hybrid_serving_example():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "hybrid_serving.py")],
                       capture_output=True, text=True, timeout=240, cwd=ROOT)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.rstrip().endswith("ok")
