"""The block-scaled 8-bit cache through the bounds-checking build
(libkvq_debug.so): every block that a kernel computes is checked against the
planes the call describes; the tests of the release build pass with it, and
the device error word stays clean (their fixture reads it at the end)."""
import os
import subprocess
import sys

import pytest

from hadamard_rotated_bit_fwht_b200 import build

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_debug_build_passes_and_stays_clean():
    lib = build.build(debug=True)
    env = dict(os.environ, KVQ_LIBRARY=lib)
    r = subprocess.run([sys.executable, "-m", "pytest", "-x", "-q", "tests/test_gpu_b8.py",
                        "-p", "no:cacheprovider", "-k", "not large_planes"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
