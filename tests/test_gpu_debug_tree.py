"""The tree attention's tests, over dense and 4-bit caches, under the bound-checking build.

It checks the looked-up rows and the pieces of the 4-bit kernel; the tests in the child process also assert a clean status word
where nothing is wrong."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_tree_attention_under_the_bound_checking_build():
    from sparse_compressed_attention_gb300 import build
    env = dict(os.environ, V4ATTN_LIB=build.build(debug=True))
    probe = subprocess.run([sys.executable, "-c", "import sparse_compressed_attention_gb300 as V; print(V.v4_build_info())"], cwd=ROOT,
                           env=env, capture_output=True, text=True, timeout=300)
    assert "V4_DEBUG" in probe.stdout, probe.stdout + probe.stderr
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_gpu_q4.py", "tests/test_gpu_tree.py", "tests/test_gpu_cache_calls.py",
                        "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=1800)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout
