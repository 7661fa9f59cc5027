"""Rows that lie past 2^31 elements of their buffer: the same bits as the rows by
themselves."""
import pytest
import torch

from w8a8_gemm_b200 import binding as B

from test_gpu_lora import _problem

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
M, LD = 33100, 65536      # 2.17e9 elements, 4.3 GB


def _far(t, buffer, at):
    """t's rows as columns `at` .. of the wide buffer."""
    view = buffer[:, at:at + t.shape[1]]
    view.copy_(t)
    return view


@pytest.mark.parametrize("spread", ["runs", "scattered"])
def test_rows_past_32_bits(spread):
    K, N, R, L = 64, 136, 16, 3
    p = _problem(M, K, N, R, L, seed=1, spread=spread)
    w = (p["A"], p["B"], p["scale"], B.sq_lora_plan(p["ids"], L))
    wide = torch.empty(M, LD, dtype=BF, device="cuda")
    assert (M - 1) * LD > 2 ** 31
    x, base = _far(p["x"], wide, 8), _far(p["base"], wide, 8192)
    dy, dxb = _far(p["dy"], wide, 16384), _far(p["dx_base"], wide, 65000)
    y, t = B.sq_lora_forward(p["x"], *w, p["base"])
    want = B.sq_lora_backward(p["dy"], p["x"], t, *w, p["dx_base"])
    assert torch.equal(B.sq_lora_forward(x, *w, base, y=base)[0], y)
    got = B.sq_lora_backward(dy, x, t, *w, dxb, dx=dxb)
    assert all(torch.equal(a, b) for a, b in zip(want, got))

    pos = torch.arange(M, dtype=torch.int32, device="cuda")
    inv = torch.rand(16, device="cuda")
    want = B.sq_rope_forward(p["x"], pos, inv, 32)
    assert torch.equal(B.sq_rope_forward(x, pos, inv, 32, out=wide[:, 32768:32832]), want)

    g, b = p["A"][0, 0], p["A"][0, 1]
    h, far = p["x"].view(1, M, K), x.unsqueeze(0)
    y, mean, rstd = B.sq_group_norm_forward(h, 8, g, b, act=B.SQ_ACT_SILU)
    out = wide[:, 40000:40000 + K].unsqueeze(0)
    for u, v in zip(B.sq_group_norm_forward(far, 8, g, b, act=B.SQ_ACT_SILU, y=out), (y, mean, rstd)):
        assert torch.equal(u, v)
    dh = p["dx_base"].view(1, M, K)
    want = B.sq_group_norm_backward(dh, h, 8, g, b, mean, rstd, act=B.SQ_ACT_SILU)
    d = _far(p["dx_base"], wide, 48000).unsqueeze(0)
    got = B.sq_group_norm_backward(d, far, 8, g, b, mean, rstd, act=B.SQ_ACT_SILU, dx=d)
    assert all(torch.equal(u, v) for u, v in zip(got, want))

    wq, s_w = torch.ones(N, K, dtype=torch.int8, device="cuda"), torch.ones(1, N, device="cuda")
    want = B.sq_dualscale_seglinear_input_grad(p["dy"], wq, s_w, None, B.Segments())
    got = B.sq_dualscale_seglinear_input_grad(dy, wq, s_w, None, B.Segments(),
                                              dx=wide[:, 56000:56000 + K])
    assert torch.equal(got, want)
    assert B.sq_get_device_status() == B.SQ_OK
