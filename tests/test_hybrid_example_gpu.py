"""The hybrid serving example end to end: recurrent layers, the paged
key/value cache, drafts rolled back, and pages handed back."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "hybrid_serving.py")], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    assert r.stdout.count("device status 0") == 2
