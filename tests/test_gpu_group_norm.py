"""Channels-last group norm with an activation (sq_group_norm_forward,
sq_group_norm_backward) against the 64-bit formulas."""
import pytest
import torch

from w8a8_gemm_b200 import binding as B

import ops_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

CASES = [  # B, S, C, G
    (1, 1, 8, 1), (1, 1, 64, 8), (2, 3, 24, 24), (1, 7, 40, 5), (3, 64, 320, 32), (1, 391, 1280, 32),
    (2, 1000, 96, 3), (1, 5000, 128, 32), (2, 77, 2560, 32), (1, 9, 8192, 1024), (5, 130, 512, 1),
    (1, 20011, 16, 2), (64, 5, 64, 4),
]


def _inputs(Bn, S, C, seed, mean=0.0, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda")

    x = (randn(Bn, S, C) * std * torch.exp(0.5 * randn(C)) + mean + randn(C)).to(BF)
    return x, (1 + 0.3 * randn(C)).to(BF), (0.3 * randn(C)).to(BF), randn(Bn, S, C).to(BF)


@pytest.mark.parametrize("act", [B.SQ_ACT_NONE, B.SQ_ACT_SILU, B.SQ_ACT_GELU])
@pytest.mark.parametrize("Bn,S,C,G", CASES)
def test_forward_and_backward(Bn, S, C, G, act):
    x, gamma, beta, dy = _inputs(Bn, S, C, seed=S + C)
    y, mean, rstd = B.sq_group_norm_forward(x, G, gamma, beta, eps=1e-4, act=act)
    (yr, ye), (mr, me), (rr, re) = ref.group_norm_forward(x, G, gamma, beta, 1e-4, act)
    ref.check(mean, mr, me, "mean")
    ref.check(rstd, rr, re, "rstd")
    ref.check(y, yr, ye, "y")
    for grads in (BF, F32):
        dx, dgamma, dbeta = B.sq_group_norm_backward(dy, x, G, gamma, beta, mean, rstd, act=act,
                                                     grad_dtype=grads)
        want = ref.group_norm_backward(dy, x, G, gamma, beta, mean, rstd, act)
        assert dgamma.dtype == dbeta.dtype == grads
        for name, got in (("dx", dx), ("dgamma", dgamma), ("dbeta", dbeta)):
            ref.check(got, *want[name], name)


@pytest.mark.parametrize("mean,std", [(1000.0, 8.0), (-30.0, 0.2), (0.0, 1e-6), (3e4, 100.0)])
def test_mean_far_above_the_deviation(mean, std):
    x, gamma, beta, _ = _inputs(2, 600, 64, seed=5)
    x = (mean + std * torch.randn(2, 600, 64, device="cuda",
                                  generator=torch.Generator("cuda").manual_seed(1))).to(BF)
    x[0, 0] = 0.0          # an outlier in the first row of a chunk
    y, m, r = B.sq_group_norm_forward(x, 8, gamma, beta, eps=1e-6, act=B.SQ_ACT_SILU)
    (yr, ye), (mr, me), (rr, re) = ref.group_norm_forward(x, 8, gamma, beta, 1e-6, B.SQ_ACT_SILU)
    ref.check(m, mr, me, "mean")
    ref.check(r, rr, re, "rstd")
    ref.check(y, yr, ye, "y")


def test_constant_input_gives_beta():
    x = torch.full((2, 50, 32), 3.5, dtype=BF, device="cuda")
    beta = torch.arange(32, device="cuda").to(BF)
    y, mean, rstd = B.sq_group_norm_forward(x, 4, None, beta, eps=1e-5)
    assert (mean == 3.5).all()
    assert torch.equal(y, beta.expand_as(y))


def test_without_parameters_strides_and_in_place():
    Bn, S, C, G = 2, 90, 48, 6
    x, _, _, dy = _inputs(Bn, S, C, seed=8)
    wide = torch.full((Bn, S, C + 16), float("nan"), dtype=BF, device="cuda")
    wide[..., 8:8 + C] = x
    view = wide[..., 8:8 + C]
    (yr, ye), _, _ = ref.group_norm_forward(x, G, None, None, 1e-5, B.SQ_ACT_GELU)
    y, mean, rstd = B.sq_group_norm_forward(view, G, None, None, act=B.SQ_ACT_GELU)
    ref.check(y, yr, ye, "y")
    want = ref.group_norm_backward(dy, x, G, None, None, mean, rstd, B.SQ_ACT_GELU)
    g = dy.clone()
    dx, dgamma, dbeta = B.sq_group_norm_backward(g, view, G, None, None, mean, rstd,
                                                 act=B.SQ_ACT_GELU, dx=g)
    assert dgamma is None and dbeta is None and dx is g
    ref.check(dx, *want["dx"], "dx")
    y2, _, _ = B.sq_group_norm_forward(view, G, None, None, act=B.SQ_ACT_GELU, y=view)
    assert torch.equal(y2, y)
    assert torch.isnan(wide[..., :8]).all() and torch.isnan(wide[..., 8 + C:]).all()


def test_parameter_gradients_only_no_samples_and_capture():
    x, gamma, beta, dy = _inputs(2, 300, 64, seed=11)
    y, mean, rstd = B.sq_group_norm_forward(x, 8, gamma, beta)
    full = B.sq_group_norm_backward(dy, x, 8, gamma, beta, mean, rstd)
    part = B.sq_group_norm_backward(dy, x, 8, gamma, beta, mean, rstd, need_dx=False)
    assert part[0] is None
    assert torch.equal(full[1], part[1]) and torch.equal(full[2], part[2])
    e = torch.empty(0, 5, 64, dtype=BF, device="cuda")
    y0, m0, r0 = B.sq_group_norm_forward(e, 8, gamma, beta)
    assert y0.shape == (0, 5, 64)
    _, dg, db = B.sq_group_norm_backward(e, e, 8, gamma, beta, m0, r0)
    assert (dg == 0).all() and (db == 0).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y1, m1, r1 = B.sq_group_norm_forward(x, 8, gamma, beta)
        got = B.sq_group_norm_backward(dy, x, 8, gamma, beta, m1, r1)
    graph.replay()
    for u, v in zip(full, got):
        assert torch.equal(u, v)
