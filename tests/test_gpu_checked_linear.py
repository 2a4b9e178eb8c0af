"""The linear layers and norms against the bounds-checked build of the library:
its checks raise no false alarm and change no result."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_linear_layers_and_norms_against_the_checked_build():
    from nvfp4_precision_b200 import build
    build.build(checked=True)
    env = dict(os.environ, FP4ATTN_BOUNDS_CHECK="1")
    tests = ["tests/test_gpu_linear.py", "tests/test_gpu_linear_backward.py", "tests/test_gpu_norm.py"]
    code = ("import sys, pytest\n"
            "from nvfp4_precision_b200 import fp4attn\n"
            "assert fp4attn.LIB_PATH.endswith('libfp4attn_checked.so'), fp4attn.LIB_PATH\n"
            f"sys.exit(pytest.main({tests!r} + ['-q', '-m', 'gpu', '-p', 'no:cacheprovider']))\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
