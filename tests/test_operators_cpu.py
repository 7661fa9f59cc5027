"""The operators around the quantized linear, without a GPU: their refusals, the
rotary frequencies, and the 64-bit reference gradients against differences."""
import ctypes
import math

import pytest
import torch

from w8a8_gemm_b200 import binding as B
from w8a8_gemm_b200 import build as sqbuild

import ops_ref as ref

INVALID, UNSUPPORTED, ALIGNMENT = -1, -2, -3
FAKE = 0x10000   # 256-byte aligned, never dereferenced: validation fails first
F64 = torch.float64


@pytest.fixture(scope="module")
def L():
    sqbuild.build()
    return B.lib()


def _call(entry, good, **changes):
    """entry with the arguments of `good` (an ordered dict), some of them changed."""
    assert set(changes) <= set(good), changes
    return entry(*{**good, **changes}.values(), None)


def test_lora_refusals(L):
    assert L.sq_lora_plan_bytes(-1, 2) == 0 and L.sq_lora_plan_bytes(8, 0) == 0
    assert L.sq_lora_plan_bytes(8, 1025) == 0 and L.sq_lora_plan_bytes(2 ** 24 + 1, 1) == 0
    assert L.sq_lora_plan_bytes(0, 1) > 0
    need = L.sq_lora_workspace_bytes(4, 8, 2, 0)
    assert need > 0 and L.sq_lora_workspace_bytes(4, 8, 2, 1) == 3 * need
    for bad in ((4, 12, 2, 0), (4, 8, 0, 0), (4, 8, 2, 2), (-1, 8, 2, 0), (4, 136, 2, 0)):
        assert L.sq_lora_workspace_bytes(*bad) == 0
    plan = dict(adapter=FAKE, M=4, L=2, plan=FAKE)
    for bad in (dict(adapter=None), dict(plan=None), dict(M=-1), dict(L=0), dict(L=1025)):
        assert _call(L.sq_lora_plan, plan, **bad) == INVALID, bad
    assert _call(L.sq_lora_plan, plan, adapter=FAKE + 2) == ALIGNMENT
    assert _call(L.sq_lora_plan, plan, plan=FAKE + 4) == ALIGNMENT

    fwd = dict(x=FAKE, ldx=64, A=FAKE, B=FAKE, scale=FAKE, plan=FAKE, base=FAKE, ldbase=72,
               y=2 * FAKE, ldy=72, out=0, t=FAKE, workspace=FAKE, bytes=need, M=4, N=72, K=64, R=8, L=2)
    for bad in (dict(x=None), dict(A=None), dict(B=None), dict(scale=None), dict(plan=None),
                dict(y=None), dict(t=None), dict(workspace=None), dict(bytes=need - 1), dict(out=2), dict(ldx=56), dict(ldy=64),
                dict(ldbase=64), dict(M=-1), dict(N=0), dict(K=0), dict(R=0), dict(L=0),
                dict(ldx=2 ** 43), dict(base=2 * FAKE, ldbase=80), dict(N=2 ** 20 + 8)):
        assert _call(L.sq_lora_forward, fwd, **bad) == INVALID, bad
    for bad in (dict(R=4), dict(R=136)):
        assert _call(L.sq_lora_forward, fwd, **bad) == UNSUPPORTED, bad
    for bad in (dict(R=12), dict(K=60), dict(N=68), dict(ldx=68), dict(x=FAKE + 2),
                dict(A=FAKE + 8), dict(workspace=FAKE + 8), dict(y=FAKE + 8), dict(t=FAKE + 8), dict(scale=FAKE + 2),
                dict(plan=FAKE + 4), dict(base=FAKE + 8)):
        assert _call(L.sq_lora_forward, fwd, **bad) == ALIGNMENT, bad
    assert _call(L.sq_lora_forward, fwd, M=0, x=None, y=None, base=None, t=None) == 0

    bwd = dict(dy=FAKE, lddy=72, x=FAKE, ldx=64, t=FAKE, A=FAKE, B=FAKE, scale=FAKE, plan=FAKE,
               dx_base=FAKE, ldbase=64, dx=2 * FAKE, lddx=64, dA=FAKE, dB=FAKE, grads=0,
               workspace=FAKE, bytes=need, M=4, N=72, K=64, R=8, L=2)
    for bad in (dict(dy=None), dict(x=None), dict(t=None), dict(workspace=None), dict(bytes=need - 1), dict(dA=None),
                dict(dB=None), dict(dx=None), dict(grads=5), dict(lddy=64), dict(ldx=56),
                dict(lddx=56), dict(ldbase=56), dict(dx_base=2 * FAKE, ldbase=72)):
        assert _call(L.sq_lora_backward, bwd, **bad) == INVALID, bad
    for bad in (dict(dA=FAKE + 2), dict(workspace=FAKE + 4), dict(dx=FAKE + 8), dict(lddy=76)):
        assert _call(L.sq_lora_backward, bwd, **bad) == ALIGNMENT, bad
    # nothing asked for: nothing done, no device needed
    assert _call(L.sq_lora_backward, bwd, dx=None, dx_base=None, dA=None, dB=None) == 0


def test_rope_refusals(L):
    def pairs(*n):
        return (ctypes.c_int32 * len(n))(*n)

    good = dict(x=FAKE, ldx=128, out=2 * FAKE, ldo=128, dtype=0, pos=FAKE, f=FAKE,
                axis_pairs=pairs(8, 8), axes=2, factor=1.0, M=3, H=2, D=64, rot=32, layout=0)
    for call in (L.sq_rope_forward, L.sq_rope_backward):
        for bad in (dict(x=None), dict(out=None), dict(pos=None), dict(f=None), dict(dtype=3),
                    dict(layout=2), dict(rot=0), dict(rot=33), dict(rot=66), dict(D=0),
                    dict(D=1032), dict(H=0), dict(M=-1), dict(axes=0), dict(axes=5),
                    dict(axis_pairs=None), dict(axis_pairs=pairs(8, 9)),
                    dict(axis_pairs=pairs(8, 7)), dict(axis_pairs=pairs(-1, 17)), dict(ldx=120),
                    dict(ldo=120), dict(out=FAKE, ldo=136), dict(factor=math.inf),
                    dict(factor=math.nan), dict(H=2 ** 20)):
            assert _call(call, good, **bad) == INVALID, bad
        for bad in (dict(D=60), dict(ldx=132), dict(x=FAKE + 8), dict(pos=FAKE + 2),
                    dict(f=FAKE + 2)):
            assert _call(call, good, **bad) == ALIGNMENT, bad
        assert _call(call, good, M=0, x=None, out=None, pos=None) == 0


def test_group_norm_refusals(L):
    size = L.sq_group_norm_workspace_bytes
    assert size(2, 100, 64, 8) > 0 and size(0, 100, 64, 8) == 0
    for bad in ((-1, 1, 8, 1), (65536, 1, 8, 1), (1, 0, 8, 1), (1, 1, 4, 1), (1, 1, 12, 1),
                (1, 1, 8200, 1), (1, 1, 64, 7), (1, 1, 64, 0), (1, 1, 8192, 2048)):
        assert size(*bad) == 0
    ws = size(2, 100, 64, 8)
    fwd = dict(x=FAKE, ldx=64, B=2, S=100, C=64, G=8, gamma=FAKE, beta=FAKE, eps=1e-5, act=1,
               y=FAKE, ldy=64, mean=FAKE, rstd=FAKE, workspace=FAKE, bytes=ws)
    for bad in (dict(x=None), dict(y=None), dict(mean=None), dict(rstd=None),
                dict(workspace=None), dict(bytes=ws - 1), dict(eps=-1.0), dict(eps=math.nan),
                dict(eps=math.inf), dict(act=3), dict(act=-1), dict(G=7), dict(S=0), dict(B=-1),
                dict(ldx=56), dict(ldy=72), dict(C=8200)):
        assert _call(L.sq_group_norm_forward, fwd, **bad) == INVALID, bad
    for bad in (dict(x=FAKE + 2), dict(ldx=68), dict(gamma=FAKE + 1), dict(mean=FAKE + 2),
                dict(workspace=FAKE + 8)):
        assert _call(L.sq_group_norm_forward, fwd, **bad) == ALIGNMENT, bad
    assert _call(L.sq_group_norm_forward, fwd, B=0, x=None, y=None) == 0
    bwd = dict(dy=FAKE, lddy=64, x=2 * FAKE, ldx=64, B=2, S=100, C=64, G=8, gamma=FAKE, beta=FAKE,
               mean=FAKE, rstd=FAKE, act=1, dx=FAKE, lddx=64, dgamma=FAKE, dbeta=FAKE, grads=0,
               workspace=FAKE, bytes=ws)
    for bad in (dict(dy=None), dict(x=None), dict(mean=None), dict(grads=2), dict(lddx=72),
                dict(dx=2 * FAKE), dict(bytes=0), dict(act=9)):
        assert _call(L.sq_group_norm_backward, bwd, **bad) == INVALID, bad
    for bad in (dict(dgamma=FAKE + 1), dict(dbeta=FAKE + 2, grads=1), dict(dy=FAKE + 8)):
        assert _call(L.sq_group_norm_backward, bwd, **bad) == ALIGNMENT, bad
    assert _call(L.sq_group_norm_backward, bwd, dx=None, dgamma=None, dbeta=None) == 0


def test_input_grad_refusals(L):
    size = L.sq_input_grad_workspace_bytes
    assert size(100, 64) == 104 * 64 * 2
    assert size(0, 64) == size(8, 24) == size(8, 0) == size(2 ** 20 + 1, 64) == 0
    c, keep = B.Segments(B.SQ_SEG_INPUT, [0, 32, 64])._c()
    good = dict(dy=FAKE, lddy=104, wq=FAKE, s_w=FAKE, d=FAKE, seg=ctypes.byref(c), dx=2 * FAKE,
                lddx=64, M=5, N=100, K=64, workspace=FAKE, bytes=size(100, 64))
    f = L.sq_dualscale_seglinear_input_grad
    for bad in (dict(dy=None), dict(wq=None), dict(s_w=None), dict(dx=None), dict(dx=FAKE),
                dict(workspace=None), dict(bytes=size(100, 64) - 1), dict(M=-1), dict(N=0),
                dict(K=72), dict(K=96), dict(lddy=96), dict(lddx=56)):
        assert _call(f, good, **bad) == INVALID, bad
    for bad in (dict(lddy=100), dict(dy=FAKE + 8), dict(wq=FAKE + 8), dict(s_w=FAKE + 2),
                dict(workspace=FAKE + 16)):
        assert _call(f, good, **bad) in (ALIGNMENT, INVALID), bad
    assert _call(f, good, workspace=FAKE + 16) == ALIGNMENT
    assert _call(f, good, M=0, dy=None, dx=None) == 0
    bad, keep2 = B.Segments(B.SQ_SEG_INPUT, [0, 48, 64])._c()
    assert _call(f, good, seg=ctypes.byref(bad)) == UNSUPPORTED


def test_binding_refuses_what_the_library_cannot_see():
    """Types, shapes and devices, before any library call."""
    bf = torch.bfloat16
    x = torch.zeros(4, 64, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        B.sq_lora_plan(torch.zeros(4, dtype=torch.int32), 2)
    with pytest.raises(ValueError, match="CUDA"):
        B.sq_lora_forward(x, x, x, x, x, None)
    with pytest.raises(ValueError, match="CUDA"):
        B.sq_group_norm_forward(x[None], 8, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        B.sq_rope_forward(x, torch.zeros(4, dtype=torch.int32), torch.zeros(16), 32)
    with pytest.raises(ValueError, match="CUDA"):
        B.sq_dualscale_seglinear_input_grad(x, x, x, None, B.Segments())
    with pytest.raises(ValueError, match="bf16 or fp32"):
        B.sq_rope_forward(x.half(), x, x, 32)
    with pytest.raises(B.SegQuantError):
        B.sq_rope_frequencies(33)
    with pytest.raises(B.SegQuantError):
        B.sq_rope_frequencies(32, scaling=B.SQ_ROPE_SCALE_LINEAR, scale=0.5)


# ------------------------------------------------------------------ frequencies
def test_rope_frequencies():
    rot, base = 64, 10000.0
    i = torch.arange(rot // 2, dtype=F64)
    plain = base ** (-2 * i / rot)

    def close(got, want):
        assert torch.equal(got, want.float()) or float(
            ((got.double() - want) / want).abs().max()) <= 2.0 ** -24 * 1.01

    f, a = B.sq_rope_frequencies(rot, base)
    close(f, plain)
    assert a == 1.0
    f, a = B.sq_rope_frequencies(rot, base, B.SQ_ROPE_SCALE_LINEAR, 4.0)
    close(f, plain / 4)
    assert a == 1.0
    f, _ = B.sq_rope_frequencies(rot, base, B.SQ_ROPE_SCALE_NTK, 8.0)
    assert f[0] == 1.0                                      # the fastest pair stays
    assert math.isclose(float(f[-1]), float(plain[-1]) / 8, rel_tol=2.0 ** -23)  # the slowest / 8
    # by parts: fast pairs as trained, slow pairs interpolated, a ramp between
    s, orig = 16.0, 4096.0
    f, a = B.sq_rope_frequencies(rot, base, B.SQ_ROPE_SCALE_YARN, s, orig)

    def pair(turns):   # the pair that makes so many turns over the trained context
        return rot * math.log(orig / (2 * math.pi * turns)) / (2 * math.log(base))

    lo, hi = math.floor(pair(32)), math.ceil(pair(1))
    r = 1 - ((i - lo) / (hi - lo)).clamp(0, 1)
    close(f, plain * ((1 - r) / s + r))
    assert 0 < lo < hi < rot // 2
    assert torch.equal(f[:lo], plain[:lo].float())
    assert math.isclose(a, 0.1 * math.log(s) + 1, rel_tol=1e-6)
    # a context so short that both ends meet: still finite and within the two forms
    f, _ = B.sq_rope_frequencies(rot, base, B.SQ_ROPE_SCALE_YARN, s, 1.0)
    assert torch.isfinite(f).all() and (f <= plain.float()).all() and (
        f.double() >= plain / s * 0.999).all()


# -------------------------------------------- reference gradients vs differences
def _differences(f, args, which, dout, n=6, h=1e-5, seed=0):
    """Central differences of <f(args), dout> along random directions of
    args[which] -> [(direction, difference)]."""
    g = torch.Generator().manual_seed(seed)
    for _ in range(n):
        v = torch.randn(args[which].shape, generator=g, dtype=F64)
        up, dn = list(args), list(args)
        up[which], dn[which] = args[which] + h * v, args[which] - h * v
        yield v, float(((f(*up) - f(*dn)) * dout).sum()) / (2 * h)


def test_reference_gradients_against_differences():
    g = torch.Generator().manual_seed(3)

    def randn(*s):
        return torch.randn(*s, generator=g, dtype=F64)

    # adapters: rows 0..8 of two adapters, one row without
    x, A, Bm, base = randn(9, 16), randn(2, 8, 16), randn(2, 24, 8), randn(9, 24)
    scale, ids, dy = torch.tensor([0.7, -1.3]), torch.tensor([0, 1, 1, -1, 0, 1, 0, 0, 1]), randn(9, 24)

    def lora(x, A, Bm):
        return ref.lora_forward(x, A, Bm, scale, ids, base, torch.float32)[0]

    t = ref.lora_forward(x, A, Bm, scale, ids, base, torch.float32)[2]
    want = ref.lora_backward(dy, x, t, A, Bm, scale, ids, None, torch.float32)
    for which, name in ((0, "dx"), (1, "dA"), (2, "dB")):
        for v, diff in _differences(lora, (x, A, Bm), which, dy):
            assert math.isclose(float((want[name][0] * v).sum()), diff, rel_tol=1e-6, abs_tol=1e-7)

    # rotary: the backward turn is the gradient
    f = torch.tensor([1.0, 0.3, 0.02])
    pos = torch.tensor([[0], [5], [-70], [1000]])
    z, dz = randn(4, 16), randn(4, 16)
    for layout in (0, 1):
        def turn(z):
            return ref.rope(z, pos, f, 8, layout, None, 1.2, 1.0)[0]

        back = ref.rope(dz, pos, f, 8, layout, None, 1.2, -1.0)[0]
        for v, diff in _differences(turn, (z,), 0, dz):
            assert math.isclose(float((back * v).sum()), diff, rel_tol=1e-6, abs_tol=1e-7)

    # group norm with each activation
    x, gm, bt, dy = randn(2, 5, 12), randn(12), randn(12), randn(2, 5, 12)
    for kind in (0, 1, 2):
        def norm(x, gm, bt):
            return ref.group_norm_forward(x, 3, gm, bt, 1e-3, kind)[0][0]

        _, (mean, _), (rstd, _) = ref.group_norm_forward(x, 3, gm, bt, 1e-3, kind)
        want = ref.group_norm_backward(dy, x, 3, gm, bt, mean, rstd, kind)
        for which, name in ((0, "dx"), (1, "dgamma"), (2, "dbeta")):
            for v, diff in _differences(norm, (x, gm, bt), which, dy):
                assert math.isclose(float((want[name][0] * v).sum()), diff, rel_tol=1e-5,
                                    abs_tol=1e-6)

    # input gradient: dx is the product with the dequantized weight
    w = ref.dequantized(torch.randint(-9, 9, (12, 64), generator=g), torch.rand(2, 12, generator=g),
                        torch.rand(1, 64, generator=g) + 0.5, 2, [0, 32, 64], 1)
    x, dy = randn(3, 64), randn(3, 12)
    dx = ref.input_grad(dy, w)[0]
    for v, diff in _differences(lambda x: x @ w.t(), (x,), 0, dy):
        assert math.isclose(float((dx * v).sum()), diff, rel_tol=1e-6, abs_tol=1e-7)


def test_lora_outputs_over_inputs_are_refused(L):
    """The kernels of a call run side by side: an output in an input's place."""
    need = L.sq_lora_workspace_bytes(4, 8, 2, 0)
    fwd = dict(x=FAKE, ldx=64, A=FAKE, B=FAKE, scale=FAKE, plan=FAKE, base=None, ldbase=0,
               y=FAKE, ldy=64, out=0, t=FAKE, workspace=FAKE, bytes=need, M=4, N=64, K=64, R=8, L=2)
    assert _call(L.sq_lora_forward, fwd) == INVALID
    bwd = dict(dy=FAKE, lddy=64, x=2 * FAKE, ldx=64, t=FAKE, A=FAKE, B=FAKE, scale=FAKE, plan=FAKE,
               base=None, ldbase=0, dx=FAKE, lddx=64, dA=FAKE, dB=FAKE, grads=0, workspace=FAKE,
               bytes=need, M=4, N=64, K=64, R=8, L=2)
    assert _call(L.sq_lora_backward, bwd) == INVALID
    assert _call(L.sq_lora_backward, bwd, dx=2 * FAKE) == INVALID
