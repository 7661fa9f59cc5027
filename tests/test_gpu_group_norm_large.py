"""Group norm with parameters so large that the activations are flat:
sq_group_norm_backward against the 64-bit formulas."""
import pytest
import torch

from w8a8_gemm_b200 import binding as B

import ops_ref as ref
from test_gpu_group_norm_values import _gen, _randn

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("act", [B.SQ_ACT_SILU, B.SQ_ACT_GELU])
@pytest.mark.parametrize("exponent", [20, 42, 50, 60])
def test_activations_of_large_values_are_flat(exponent, act):
    """v up to 2^62, whose cube is past the largest fp32 number: the derivative is
    1 above and 0 below."""
    Bn, S, C, G = 1, 200, 64, 4
    g = _gen(exponent)
    x, dy = _randn(g, Bn, S, C).to(BF), _randn(g, Bn, S, C).to(BF)
    gamma = torch.full((C,), 2.0 ** exponent, dtype=BF, device="cuda")
    y, mean, rstd = B.sq_group_norm_forward(x, G, gamma, None, act=act)
    (yr, ye), _, _ = ref.group_norm_forward(x, G, gamma, None, 1e-5, act)
    ref.check(y, yr, ye, "y")
    want = ref.group_norm_backward(dy, x, G, gamma, None, mean, rstd, act)
    dx, dgamma, _ = B.sq_group_norm_backward(dy, x, G, gamma, None, mean, rstd, act=act)
    ref.check(dx, *want["dx"], "dx")
    ref.check(dgamma, *want["dgamma"], "dgamma")
