"""Group norm where the mean is far above the deviation, and with infinities:
sq_group_norm_forward and _backward against the 64-bit formulas."""
import pytest
import torch

from w8a8_gemm_b200 import binding as B

import ops_ref as ref

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
SIZES = [(2, 50, 32, 4), (1, 391, 1280, 32), (3, 1, 64, 8), (1, 4100, 48, 3), (2, 20000, 16, 2),
         (1, 9, 8192, 1024)]


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _parameters(g, C, with_beta):
    gamma = (1 + 0.5 * _randn(g, C)).to(BF)
    return gamma, (2 * _randn(g, C)).to(BF) if with_beta else None


@pytest.mark.parametrize("eps", [1e-5, 1e-6])
@pytest.mark.parametrize("with_beta", [False, True])
@pytest.mark.parametrize("Bn,S,C,G", SIZES)
def test_constant_groups_give_beta(Bn, S, C, G, with_beta, eps):
    """The deviation from the mean is zero whatever the value: y is act(beta) and
    the mean is the value itself."""
    g = _gen(S + C)
    value = (_randn(g, Bn, G) * torch.exp(4 * _randn(g, Bn, G))).to(BF)
    x = value.repeat_interleave(C // G, 1)[:, None].expand(Bn, S, C).contiguous()
    gamma, beta = _parameters(g, C, with_beta)
    want = torch.zeros(C, dtype=BF, device="cuda") if beta is None else beta
    y, mean, rstd = B.sq_group_norm_forward(x, G, gamma, beta, eps=eps)
    assert torch.equal(mean, value.float())
    assert torch.equal(y, want.expand_as(y))
    # a double square root and quotient, rounded to fp32; eps is an fp32 argument
    r = torch.full_like(rstd, 1.0, dtype=F64) / torch.tensor(eps, dtype=F32).to(F64).sqrt()
    ref.check(rstd, r, 2.0 ** -50 * r, "rstd")
    y, _, _ = B.sq_group_norm_forward(x, G, gamma, beta, eps=eps, act=B.SQ_ACT_SILU)
    v = want.to(F64)
    ref.check(y, ref.act(v, B.SQ_ACT_SILU)[0].expand_as(y),
              ref.ACT_EVAL * (1 + v.abs()).expand_as(y), "y with SiLU")


@pytest.mark.parametrize("Bn,S,C,G", SIZES)
def test_few_values_beside_a_constant(Bn, S, C, G):
    """Groups of one value and a few of the next bf16 one: y from the call's own
    statistics within the roundings of (x - mean) rstd gamma + beta (the difference,
    rstd gamma, and the result of the multiply-add), and the statistics within
    theirs."""
    g = _gen(S * C)
    value = (256 * torch.exp2(torch.randint(-4, 5, (Bn, 1, G, 1), generator=g, device="cuda")))
    step = torch.rand(Bn, S, G, C // G, generator=g, device="cuda") < 3.0 / (S * C // G)
    z = torch.where(step, value * (1 + 2.0 ** -7), value.expand_as(step)).float()
    x = z.to(BF).reshape(Bn, S, C)
    gamma, beta = _parameters(g, C, True)
    y, mean, rstd = B.sq_group_norm_forward(x, G, gamma, beta, eps=1e-5)
    mu, rs = ref._per_channel(mean, C), ref._per_channel(rstd, C)
    gm, bt = gamma.to(F64), beta.to(F64)
    p = (x.to(F64) - mu) * rs * gm
    ref.check(y, p + bt, 2.0 ** -22 * p.abs() + 2.0 ** -23 * (p + bt).abs(), "y")

    # A thread's mean of up to 32 rows rounds once, as do its joins (fewer than
    # four here), the threads' of a channel, the channels' and the result: 2^-20 of
    # the value.  What is summed besides are distances within the group, at most
    # 2^8 in a row: 2^-15 of the largest.
    xg = x.to(F64).reshape(Bn, S, G, C // G)
    exact = xg.mean((1, 3))
    spread = xg.amax((1, 3)) - xg.amin((1, 3))
    em = 2.0 ** -20 * exact.abs() + 2.0 ** -15 * spread
    ref.check(mean, exact, em, "mean")
    var = (xg - exact[:, None, :, None]).square().mean((1, 3))
    r = 1 / (var + 1e-5).sqrt()
    # distances between means are off by twice em: squares by 4 em sqrt(var) + 4 em^2
    ev = 2.0 ** -14 * var + 4 * em * var.sqrt() + 4 * em * em
    ref.check(rstd, r, r * ev * r * r, "rstd")


@pytest.mark.parametrize("act", [B.SQ_ACT_NONE, B.SQ_ACT_SILU, B.SQ_ACT_GELU])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_infinities_stay_in_their_group(bad, act):
    Bn, S, C, G = 2, 300, 96, 6
    g = _gen(3)
    x, dy = _randn(g, Bn, S, C).to(BF), _randn(g, Bn, S, C).to(BF)
    gamma, beta = _parameters(g, C, True)
    y, mean, rstd = B.sq_group_norm_forward(x, G, gamma, beta, act=act)
    clean = B.sq_group_norm_backward(dy, x, G, gamma, beta, mean, rstd, act=act)
    z = x.clone()
    z[1, 77, 40] = bad                       # group 2 of the second sample
    y2, mean2, rstd2 = B.sq_group_norm_forward(z, G, gamma, beta, act=act)
    grads = B.sq_group_norm_backward(dy, z, G, gamma, beta, mean2, rstd2, act=act)
    hit = torch.zeros(Bn, G, dtype=torch.bool, device="cuda")
    hit[1, 2] = True
    assert not torch.isfinite(mean2[hit]).any() and torch.isnan(rstd2[hit]).all()
    assert torch.equal(mean2[~hit], mean[~hit]) and torch.equal(rstd2[~hit], rstd[~hit])
    where = hit.repeat_interleave(C // G, 1)[:, None].expand_as(y)
    for got, want in ((y2, y), (grads[0], clean[0])):
        assert torch.isnan(got[where]).all() and torch.equal(got[~where], want[~where])
    rest = ~hit[1].repeat_interleave(C // G)
    for got, want in zip(grads[1:], clean[1:]):
        assert torch.equal(got[rest], want[rest])
