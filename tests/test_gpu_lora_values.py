"""Adapters: infinities in the forms that keep 24 bits, the buffers of a whole
prompt in place, and single rows with any stride, against the 64-bit formulas."""
import pytest
import torch

from w8a8_gemm_b200 import binding as B

import ops_ref as ref
from test_gpu_lora import _problem

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
INF = float("inf")


def _same_where_not_finite(got, want, name):
    """NaN where the formula has NaN, infinities of its signs, finite elsewhere."""
    assert torch.equal(torch.isnan(got), torch.isnan(want)), name
    odd = ~torch.isfinite(want) & ~torch.isnan(want)
    assert torch.equal(~torch.isfinite(got), ~torch.isfinite(want)), name
    assert torch.equal(got[odd].double(), want[odd]), name


@pytest.mark.parametrize("grads", [BF, F32])
@pytest.mark.parametrize("R", [16, 128])
def test_infinite_values_in_the_backward_pass(R, grads):
    """t has values with few bits, many bits, zeros and an infinity; dy an infinity
    of each sign."""
    M, K, N, L = 300, 128, 136, 3
    p = _problem(M, K, N, R, L, seed=4, spread="scattered")
    rows = [(p["ids"] == a).nonzero()[:, 0] for a in range(L)]
    g = torch.Generator("cuda").manual_seed(R)
    t = torch.randn(M, R, generator=g, device="cuda")
    t[:, ::4] = torch.randint(-3, 4, (M, (R + 3) // 4), generator=g, device="cuda").float()
    t[:, 1] = 2.0 ** -60
    p["dy"][rows[1][0], 7], p["dy"][rows[1][3], 9] = INF, -INF
    t[rows[0][2], 5] = -INF
    x = p["x"]
    x[rows[2][1], 11] = INF
    plan = B.sq_lora_plan(p["ids"], L)
    dA, dB, _ = B.sq_lora_backward(p["dy"], x, t, p["A"], p["B"], p["scale"], plan, None,
                                   grad_dtype=grads, need_dx=False)
    for a in range(L):
        r, c = rows[a], float(p["scale"][a])
        dy, ta = p["dy"][r].double(), t[r].double()
        terms = c * dy[:, :, None] * ta[:, None]              # sums of products, no matrix call
        _same_where_not_finite(dB[a], terms.sum(0), f"dB[{a}]")
        dt = c * (dy[:, :, None] * p["B"][a].double()[None]).sum(1)
        _same_where_not_finite(dA[a], (dt[:, :, None] * x[r].double()[:, None]).sum(0), f"dA[{a}]")


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,R", [(12, 8), (30, 64), (300, 24), (300, 128)])
def test_infinite_values_in_the_forward_pass(M, R, out):
    """Small whole numbers for x and A, so that t has few bits; an infinity in B, and
    one in x, whose t is infinite."""
    K, N, L = 64, 72, 2
    p = _problem(M, K, N, R, L, seed=6, spread="scattered", out=out)
    g = torch.Generator("cuda").manual_seed(M)
    x = torch.randint(1, 4, (M, K), generator=g, device="cuda").to(BF)
    A = torch.randint(-3, 4, (L, R, K), generator=g, device="cuda").to(BF)
    Bm, scale = p["B"].clone(), torch.tensor([0.5, -2.0], device="cuda")
    Bm[1, 5, 3], Bm[0, 9, 6] = INF, -INF
    Bm[:, 11] = Bm[:, 11].abs() + 0.25
    first = int((p["ids"] == 0).nonzero()[0, 0])
    x[first, 9] = INF
    A[0, :, 9] = A[0, :, 9].abs() + 1        # t of that row: + infinity everywhere
    plan = B.sq_lora_plan(p["ids"], L)
    y, _ = B.sq_lora_forward(x, A, Bm, scale, plan, p["base"])
    want = p["base"].double().clone()
    for a in range(L):
        r = (p["ids"] == a).nonzero()[:, 0]
        t = (x[r].double()[:, None] * A[a].double()[None]).sum(2)
        want[r] += float(scale[a]) * (t[:, None] * Bm[a].double()[None]).sum(2)
    assert float(want[first, 11]) == INF
    _same_where_not_finite(y, want, "y")


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,K,N,R,L,spread", [(6000, 1536, 2304, 64, 2, "runs"),
                                              (5003, 512, 1544, 48, 5, "mixed"),
                                              (4500, 256, 3000, 128, 3, "scattered")])
def test_a_prompt_in_place(M, K, N, R, L, spread, out):
    """Several tiles and slabs of columns a block, on the projection's own output (a
    slice of a wider buffer), and dx on the frozen layer's gradient."""
    p = _problem(M, K, N, R, L, seed=M, spread=spread, out=out)
    plan = B.sq_lora_plan(p["ids"], L)
    apart, t = B.sq_lora_forward(p["x"], p["A"], p["B"], p["scale"], plan, p["base"])
    v, e, _, _ = ref.lora_forward(p["x"], p["A"], p["B"], p["scale"], p["ids"], p["base"], out)
    ref.check(apart, v, e, "y")
    wide = torch.full((M, N + 24), 3.0, dtype=out, device="cuda")
    view = wide[:, 8:8 + N]
    view.copy_(p["base"])
    B.sq_lora_forward(p["x"], p["A"], p["B"], p["scale"], plan, view, y=view)
    assert torch.equal(view, apart)
    assert (wide[:, :8] == 3.0).all() and (wide[:, 8 + N:] == 3.0).all()

    a = (p["dy"], p["x"], t, p["A"], p["B"], p["scale"], plan)
    apart = B.sq_lora_backward(*a, p["dx_base"], grad_dtype=out)
    want = ref.lora_backward(p["dy"], p["x"], t, p["A"], p["B"], p["scale"], p["ids"],
                             p["dx_base"], out)
    for name, got in zip(("dA", "dB", "dx"), apart):
        ref.check(got, *want[name], name)
    wide = torch.full((M, K + 8), 5.0, dtype=BF, device="cuda")
    view = wide[:, :K]
    view.copy_(p["dx_base"])
    dA, dB, _ = B.sq_lora_backward(*a, view, dx=view, grad_dtype=out)
    assert all(torch.equal(u, w) for u, w in zip(apart, (dA, dB, view)))
    assert (wide[:, K:] == 5.0).all()
    assert B.sq_get_device_status() == B.SQ_OK


@pytest.mark.parametrize("M,K,N,R,L,spread", [(1825, 72, 144, 8, 4, "one"), (646, 48, 104, 8, 37, "runs"),
                                              (596, 424, 72, 16, 26, "scattered"),
                                              (300, 1000, 264, 72, 2, "mixed"),
                                              (5000, 256, 128, 128, 3, "mixed")])
def test_dx_beside_fp32_gradients_keeps_16_bits_of_dt(M, K, N, R, L, spread):
    """The bound is that of the formula with dt in fp32, its first two cut-off bf16
    terms (2^-14 at most, 8 bits each) and the sums over N and 2 R products."""
    p = _problem(M, K, N, R, L, seed=R, spread=spread)
    plan = B.sq_lora_plan(p["ids"], L)
    t = torch.randn(M, R, device="cuda", generator=torch.Generator("cuda").manual_seed(M))
    _, _, dx = B.sq_lora_backward(p["dy"], p["x"], t, p["A"], p["B"], p["scale"], plan, None,
                                  grad_dtype=F32)
    want, bound = torch.zeros(M, K, dtype=F64, device="cuda"), torch.zeros(M, K, dtype=F64,
                                                                           device="cuda")
    for a in range(L):
        r = (p["ids"] == a).nonzero()[:, 0]
        g, A, Bm, c = p["dy"][r].double(), p["A"][a].double(), p["B"][a].double(), float(p["scale"][a])
        dt = c * (g @ Bm)
        e = abs(c) * ref.ACC(N + 8) * (g.abs() @ Bm.abs()) + 2.0 ** -23 * dt.abs()
        want[r] = dt @ A
        bound[r] = (e + (2.0 ** -14 + ref.ACC(2 * R)) * (dt.abs() + e)) @ A.abs()
    ref.check(dx, want, bound, "dx")
