"""The input gradient with divisors at the ends of fp32: inverses past the largest
number, below the smallest normal one, and infinite divisors."""
import pytest
import torch

from w8a8_gemm_b200 import binding as B

import ops_ref as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("M,N,K", [(3, 64, 48), (200, 1600, 256), (600, 136, 80)])
def test_divisors_without_an_inverse(M, N, K):
    """Channel k % 8 == 3 of every second octet: a divisor of 2^-130, whose inverse
    overflows; others of 2^127 (an inverse below the normal numbers) and infinity."""
    g = torch.Generator("cuda").manual_seed(M)
    wq = torch.randint(-128, 128, (N, K), generator=g, device="cuda").to(torch.int8)
    # steps so small that the quotient by 2^-130 stays finite
    s_w = (torch.rand(1, N, generator=g, device="cuda") + 0.5) * 2.0 ** -20
    d = torch.exp(torch.randn(1, K, generator=g, device="cuda"))
    d[0, 3::16] = 2.0 ** -130
    d[0, 4::16] = 1.5 * 2.0 ** 127
    d[0, 5::16] = float("inf")
    dy = (torch.randn(M, N, generator=g, device="cuda") * 2.0 ** -20).to(BF)
    dx = B.sq_dualscale_seglinear_input_grad(dy, wq, s_w, d, B.Segments())
    w = ref.dequantized(wq.double(), s_w, d, B.SQ_SEG_NONE, None, 1)
    want, bound = ref.input_grad(dy, w)
    # bf16 below 2^-126 has steps of 2^-133
    ref.check(dx, want, bound + 2.0 ** -133 * (1 + dy.double().abs().sum(1, keepdim=True)), "dx")
    assert (dx[:, 5::16] == 0).all()
