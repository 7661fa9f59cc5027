"""Outputs over inputs, and over each other, are refused before anything is
launched; the test of two buffers (csrc/spans.h) against all of their bytes."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from w8a8_gemm_b200 import binding as B
from w8a8_gemm_b200 import build as sqbuild

INVALID = -1
SHIM = """
#include "spans.h"
extern "C" int shared(uintptr_t a, int64_t ar, int64_t ab, int64_t ap, uintptr_t b, int64_t br,
                      int64_t bb, int64_t bp) {
  return sq::overlap(sq::Span(reinterpret_cast<void *>(a), ar, ab, ap),
                     sq::Span(reinterpret_cast<void *>(b), br, bb, bp));
}
"""


def test_two_buffers_against_all_of_their_bytes(tmp_path):
    src, lib = tmp_path / "spans.cpp", tmp_path / "spans.so"
    src.write_text(SHIM)
    subprocess.run([shutil.which("g++") or "g++", "-std=c++17", "-shared", "-fPIC", "-O1",
                    f"-I{sqbuild.CSRC}", str(src), "-o", str(lib)], check=True)
    f = ctypes.CDLL(os.fspath(lib)).shared
    f.argtypes = [ctypes.c_size_t] + [ctypes.c_int64] * 3 + [ctypes.c_size_t] + [ctypes.c_int64] * 3
    rng = random.Random(1)
    seen = [0, 0]
    for _ in range(20000):
        pitch = rng.randint(1, 12)
        one = rng.random() < 0.4
        a = (rng.randint(1, 60), rng.randint(0, 6), rng.randint(1, pitch), pitch)
        n = rng.randint(1, 20)
        b = ((rng.randint(1, 60), 1, n, n) if one else
             (rng.randint(1, 60), rng.randint(0, 6), rng.randint(1, pitch), pitch))
        if rng.random() < 0.5:
            a, b = b, a
        bytes_of = [{at + i * p + j for i in range(r) for j in range(n)} for at, r, n, p in (a, b)]
        want = bool(bytes_of[0] & bytes_of[1])
        assert bool(f(*a, *b)) == want, (a, b)
        seen[want] += 1
    assert min(seen) > 1000
    assert f(0, 4, 8, 8, 1, 4, 8, 8) == 0                     # an absent buffer


# ------------------------------------------------------------------- refusals
# Addresses that are never dereferenced: every call here is refused.
def at(i):
    return 0x10000000 * (i + 1)


def _refused(entry, good, cases):
    for name, changes in cases.items():
        assert set(changes) <= set(good), name
        assert entry(*{**good, **changes}.values(), None) == INVALID, name


@pytest.fixture(scope="module")
def L():
    sqbuild.build()
    return B.lib()


def test_adapters(L):
    M, N, K, R, n = 40, 72, 64, 8, 2
    ws = L.sq_lora_workspace_bytes(M, R, n, 1)
    fwd = dict(x=at(0), ldx=64, A=at(1), B=at(2), scale=at(3), plan=at(4), base=at(5), ldbase=72,
               y=at(6), ldy=72, out=1, t=at(7), workspace=at(8), bytes=ws, M=M, N=N, K=K, R=R, L=n)
    inside = 16 * 8          # bytes into a buffer
    _refused(L.sq_lora_forward, fwd, {
        "y in x": dict(y=at(0) + inside), "y over A": dict(y=at(1)), "y over B": dict(y=at(2)),
        "y beside scale": dict(y=at(3) - inside), "y over plan": dict(y=at(4)),
        "y in base": dict(y=at(5) + 4 * 72), "t over y": dict(t=at(6)), "t over A": dict(t=at(1)),
        "t in x": dict(t=at(0) + inside), "workspace over t": dict(workspace=at(7)),
        "workspace over plan": dict(workspace=at(4)), "workspace over base": dict(workspace=at(5)),
        # columns of one wider buffer: eight in common
        "y beside x": dict(x=at(0), ldx=256, y=at(0) + 56 * 2, ldy=128, base=None, ldbase=0, out=1),
        "y and base": dict(base=at(5), ldbase=160, y=at(5) + 64 * 4, ldy=160)})
    bwd = dict(dy=at(0), lddy=72, x=at(1), ldx=64, t=at(2), A=at(3), B=at(4), scale=at(5),
               plan=at(6), dx_base=at(7), ldbase=64, dx=at(8), lddx=64, dA=at(9), dB=at(10), grads=0,
               workspace=at(11), bytes=ws, M=M, N=N, K=K, R=R, L=n)
    over = {f"{o} over {k}": {o: bwd[k] + inside * (k != "scale")}
            for o in ("dA", "dB", "dx") for k in ("dy", "x", "t", "A", "B", "scale", "plan",
                                                  "dx_base", "dx", "workspace") if o != k}
    _refused(L.sq_lora_backward, bwd, {
        **over, "dA over dB": dict(dA=at(10) + inside), "workspace over A": dict(workspace=at(3)),
        "dA over A, no dx": dict(dx=None, dx_base=None, dA=at(3)),
        "dA over A, no rows": dict(M=0, dA=at(3))})
    _refused(L.sq_lora_plan, dict(adapter=at(0), M=M, L=n, plan=at(1)),
             {"plan over adapter": dict(plan=at(0))})


def test_rotary(L):
    good = dict(x=at(0), ldx=128, out=at(1), ldo=128, dtype=0, pos=at(2), f=at(3), axis_pairs=None,
                axes=1, factor=1.0, M=9, H=2, D=64, rot=32, layout=0)
    for call in (L.sq_rope_forward, L.sq_rope_backward):
        _refused(call, good, {
            "a row on": dict(out=at(0) + 256), "eight columns on": dict(out=at(0) + 16),
            "out over positions": dict(out=at(2)), "out over frequencies": dict(out=at(3)),
            "positions in out": dict(pos=at(1) + 5 * 256), "one row": dict(M=1, out=at(0) + 16)})


def test_group_norm(L):
    Bn, S, C, G = 2, 30, 64, 8
    ws = L.sq_group_norm_workspace_bytes(Bn, S, C, G)
    fwd = dict(x=at(0), ldx=64, B=Bn, S=S, C=C, G=G, gamma=at(1), beta=at(2), eps=1e-5, act=1,
               y=at(3), ldy=64, mean=at(4), rstd=at(5), workspace=at(6), bytes=ws)
    _refused(L.sq_group_norm_forward, fwd, {
        "a row on": dict(y=at(0) + 128), "y over gamma": dict(y=at(1)), "y over beta": dict(y=at(2)),
        "mean over y": dict(mean=at(3)), "mean over rstd": dict(mean=at(5)),
        "rstd over x": dict(rstd=at(0)), "mean over gamma": dict(mean=at(1)),
        "workspace over x": dict(workspace=at(0)), "workspace over mean": dict(workspace=at(4))})
    bwd = dict(dy=at(0), lddy=64, x=at(1), ldx=64, B=Bn, S=S, C=C, G=G, gamma=at(2), beta=at(3),
               mean=at(4), rstd=at(5), act=1, dx=at(6), lddx=64, dgamma=at(7), dbeta=at(8), grads=0,
               workspace=at(9), bytes=ws)
    over = {f"{o} over {k}": {o: bwd[k]} for o in ("dgamma", "dbeta", "workspace")
            for k in ("dy", "x", "gamma", "beta", "mean", "rstd", "dx")}
    _refused(L.sq_group_norm_backward, bwd, {
        **over, "dx in dy": dict(dx=at(0) + 128), "dx over x": dict(dx=at(1) + 128),
        "dx over gamma": dict(dx=at(2)), "dx over mean": dict(dx=at(4)),
        "dgamma over dbeta": dict(dgamma=at(8)), "no samples": dict(B=0, dgamma=at(2)), "workspace over dbeta": dict(workspace=at(8))})


def test_input_gradient(L):
    ws = L.sq_input_grad_workspace_bytes(104, 64)
    good = dict(dy=at(0), lddy=104, wq=at(1), s_w=at(2), d=at(3), seg=None, dx=at(4), lddx=64, M=20,
                N=104, K=64, workspace=at(5), bytes=ws)
    _refused(L.sq_dualscale_seglinear_input_grad, good, {
        "dx in dy": dict(dx=at(0) + 208), "dx over wq": dict(dx=at(1)), "dx over s_w": dict(dx=at(2)),
        "dx over d": dict(dx=at(3)), "workspace over dx": dict(workspace=at(4)),
        "workspace over dy": dict(workspace=at(0)), "workspace over wq": dict(workspace=at(1)),
        "workspace over s_w": dict(workspace=at(2)), "workspace over d": dict(workspace=at(3)),
        "columns of one buffer": dict(lddy=208, lddx=208, dx=at(0) + 96 * 2)})
