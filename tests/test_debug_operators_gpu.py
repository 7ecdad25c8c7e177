"""The operators around the attention through the library's debug variant, whose kernels
hold each global offset against its buffer's size before use: small cases, whole and
ragged, pass with no check firing.  Runs in a child process, because the variant is
chosen when the binding is imported."""
import os
import subprocess
import sys

import pytest

from tests import _gpu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_debug_library_passes_the_operators():
    _gpu.need_gpu()
    # build (or bring up to date) the debug variant; a no-op when it is current
    subprocess.run([sys.executable, os.path.join(ROOT, "static_sparse_attention_b200", "build.py"), "--debug"],
                   check=True, capture_output=True, timeout=900)
    env = dict(os.environ, RA_LIBRARY_VARIANT="debug")
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "_debug_operators_run.py")], env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "debug operators ok" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
