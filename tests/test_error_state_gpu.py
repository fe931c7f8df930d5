"""A failed CUDA call inside the library does not colour the next call."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu


def test_a_refused_launch_is_one_call_s_status():
    child = os.path.join(os.path.dirname(os.path.abspath(__file__)), "error_state_child.py")
    r = subprocess.run([sys.executable, child], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
