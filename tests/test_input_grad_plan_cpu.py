"""How the input gradient's product is cut (csrc/input_grad_plan.h), for GPUs of
any number of SMs; compiled with the host compiler, no GPU."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from w8a8_gemm_b200 import build as sqbuild

SHIM = """
#include "input_grad_plan.h"
extern "C" void plan(int64_t M, int64_t N, int64_t K, int sms, int64_t *out) {
  const sq::InputGradPlan p = sq::input_grad_plan(M, N, K, sms);
  out[0] = p.bn; out[1] = p.splits; out[2] = p.tiles; out[3] = p.clusters;
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    src, lib = d / "plan.cpp", d / "plan.so"
    src.write_text(SHIM)
    subprocess.run([shutil.which("g++") or "g++", "-std=c++17", "-shared", "-fPIC", "-O1",
                    f"-I{sqbuild.CSRC}", str(src), "-o", str(lib)], check=True)
    f = ctypes.CDLL(os.fspath(lib)).plan
    f.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int, ctypes.c_void_p]

    def call(M, N, K, sms):
        out = (ctypes.c_int64 * 4)()
        f(M, N, K, sms, out)
        return tuple(out)

    return call


def _sizes(n, seed):
    rng = random.Random(seed)
    for _ in range(n):
        yield (int(2 ** rng.uniform(0, 14)), int(2 ** rng.uniform(0, 13)),
               16 * int(2 ** rng.uniform(0, 9)))


@pytest.mark.parametrize("sms", [1, 2, 16, 29, 60, 74, 132, 144, 148, 160])
def test_shared_contractions_have_one_tile_each(plan, sms):
    """The partial sums of a shared tile take the stages' place and are added once,
    behind the tile loop: a cluster that shares a tile must have no second one."""
    shared = 0
    for M, N, K in _sizes(3000, sms):
        bn, splits, tiles, clusters = plan(M, N, K, sms)
        assert tiles == -(-M // 256) * -(-K // bn)
        assert 1 <= clusters <= tiles
        if splits > 1:
            shared += 1
            assert bn == 128 and splits in (2, 4)
            assert clusters == tiles
            assert clusters * 2 * splits <= max(sms, 0) and N > 23 * 64
        else:
            assert clusters <= max(sms // 2, 1)
    assert (shared > 0) == (sms >= 5)


def test_the_choice_on_148_sms(plan):
    for (M, N, K), want in {
            (1109, 1536, 1536): (128, 1), (8858, 6144, 1536): (256, 1), (200, 3840, 1920): (128, 4),
            (200, 1536, 1536): (128, 4), (200, 384, 768): (128, 1), (1, 1536, 128): (128, 4),
            (700, 2000, 656): (128, 2), (1025, 1600, 768): (128, 2), (257, 1536, 896): (128, 4),
            (257, 1472, 896): (128, 1)}.items():
        assert plan(M, N, K, 148)[:2] == want, (M, N, K)
