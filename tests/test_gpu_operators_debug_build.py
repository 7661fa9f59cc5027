"""The operators around the quantized linear under the bounds-checked debug
build, in a child process: the same results, and the error word clear after
every test (tests/conftest.py)."""
import os
import re
import subprocess
import sys

import pytest

from w8a8_gemm_b200 import build as sqbuild

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def test_operator_suites_pass_under_the_debug_build():
    lib = sqbuild.build(debug=True)
    env = dict(os.environ, SQ_LIBRARY=lib)
    files = ["test_gpu_lora.py", "test_gpu_rope.py", "test_gpu_group_norm.py",
             "test_gpu_input_grad.py", "test_gpu_operator_chain.py"]
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
           *[os.path.join(HERE, f) for f in files]]
    r = subprocess.run(cmd, env=env, cwd=os.path.dirname(HERE), capture_output=True, text=True,
                       timeout=900)
    tail = (r.stdout + r.stderr)[-3000:]
    assert r.returncode == 0, tail
    m = re.search(r"(\d+) passed", r.stdout)
    assert m and " failed" not in r.stdout and " skipped" not in r.stdout, tail
    assert int(m.group(1)) >= 150, tail
