"""The operators' store checks and their tests of values under the bounds-checked
debug build, in a child process (a process loads one build of the library)."""
import os
import re
import subprocess
import sys

import pytest

from w8a8_gemm_b200 import build as sqbuild

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def _run(*files):
    env = dict(os.environ, SQ_LIBRARY=sqbuild.build(debug=True))
    cmd = [sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider",
           *[os.path.join(HERE, f) for f in files]]
    r = subprocess.run(cmd, env=env, cwd=os.path.dirname(HERE), capture_output=True, text=True,
                       timeout=900)
    tail = (r.stdout + r.stderr)[-3000:]
    assert r.returncode == 0, tail
    m = re.search(r"(\d+) passed", r.stdout)
    assert m and " failed" not in r.stdout and " skipped" not in r.stdout, tail
    return int(m.group(1)), tail


def test_store_checks_of_the_operators():
    n, tail = _run("debug_build_operator_cases.py")
    assert n == 4, tail


def test_value_suites_pass_under_the_debug_build():
    n, tail = _run("test_gpu_group_norm_values.py", "test_gpu_lora_values.py",
                   "test_gpu_input_grad_divisors.py", "test_gpu_single_row.py")
    assert n >= 70, tail
