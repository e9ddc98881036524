"""The example that runs the decode operators and the junction together checks itself."""
import os
import subprocess
import sys

import pytest

from tests import test_gpu_decode as D

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

mx = D.mx


def test_decode_step_example(mx):
    r = subprocess.run([sys.executable, os.path.join("examples", "decode_step.py")], cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "decode: error" in r.stdout and "train: error" in r.stdout, r.stdout + r.stderr
