"""The debug build (every cache row checked on the device) passes the guarded cases of the norm/rotation pass
and of the 4-bit cache, in a process of its own."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


def test_debug_build_passes_the_guarded_cases():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    if not os.path.exists(os.path.join(ROOT, "sparse_top_kv_std_b200", "libstd_b200_debug.so")):
        from sparse_top_kv_std_b200 import build
        build.build(debug=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-m", "gpu", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_gpu_rope.py"), os.path.join(ROOT, "tests", "test_gpu_kv4.py")],
                       cwd=ROOT, env=dict(os.environ, STD_B200_DEBUG="1"), capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
    assert " passed" in r.stdout and "failed" not in r.stdout, r.stdout[-2000:]
