"""The debug library (libmsa_debug.so) on the calls over drafted tokens, in a process of its own.
The cases are in tests/debug_tree_cases.py."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_debug_tree_cases():
    env = dict(os.environ, MSA_LIBRARY_VARIANT="debug")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider",
                        os.path.join("tests", "debug_tree_cases.py")],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
