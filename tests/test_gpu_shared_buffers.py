"""Inputs and outputs as neighbouring columns of one buffer are no overlap; an
output that shares a byte with an input is refused."""
import pytest
import torch

from w8a8_gemm_b200 import binding as B

from test_gpu_lora import _problem

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_columns_of_one_buffer():
    M, K, N, R, L = 300, 64, 72, 8, 2
    p = _problem(M, K, N, R, L, seed=5, spread="mixed")
    w = (p["A"], p["B"], p["scale"], B.sq_lora_plan(p["ids"], L))
    y, t = B.sq_lora_forward(p["x"], *w, p["base"])
    dA, dB, dx = B.sq_lora_backward(p["dy"], p["x"], t, *w, p["dx_base"])
    wide = torch.cat([p["x"], p["base"], p["dy"], p["dx_base"]], 1).contiguous()
    cut = [wide[:, a:b] for a, b in ((0, K), (K, K + N), (K + N, K + 2 * N), (K + 2 * N, None))]
    got, u = B.sq_lora_forward(cut[0], *w, cut[1], y=cut[1])
    assert torch.equal(got, y)
    grads = B.sq_lora_backward(cut[2], cut[0], u, *w, cut[3], dx=cut[3])
    assert all(torch.equal(a, b) for a, b in zip(grads, (dA, dB, dx)))
    pos, inv = torch.arange(M, dtype=torch.int32, device="cuda"), torch.rand(16, device="cuda")
    want = B.sq_rope_forward(p["x"], pos, inv, 32)
    assert torch.equal(B.sq_rope_forward(cut[0], pos, inv, 32, out=cut[3]), want)
    h = wide[:, :K].unflatten(0, (3, 100))
    assert torch.equal(B.sq_group_norm_forward(h, 4, None, None, y=cut[3].unflatten(0, (3, 100)))[0],
                       B.sq_group_norm_forward(p["x"].view(3, 100, K), 4, None, None)[0])
    wq, s_w = torch.ones(N, K, dtype=torch.int8, device="cuda"), torch.ones(1, N, device="cuda")
    assert torch.equal(
        B.sq_dualscale_seglinear_input_grad(p["dy"], wq, s_w, None, B.Segments()),
        B.sq_dualscale_seglinear_input_grad(cut[2], wq, s_w, None, B.Segments(), dx=cut[3]))
    assert B.sq_get_device_status() == B.SQ_OK


@pytest.mark.parametrize("native", [True, False])
def test_gradients_in_the_weights_places_are_refused(native, monkeypatch):
    if not native:
        monkeypatch.setattr(B, "_native", False)
    M, K, N, R, L = 40, 64, 64, 8, 2
    p = _problem(M, K, N, R, L, seed=5, spread="one")
    w = (p["A"], p["B"], p["scale"], B.sq_lora_plan(p["ids"], L))
    _, t = B.sq_lora_forward(p["x"], *w, p["base"])
    keep = {k: v.clone() for k, v in p.items()}
    args = (p["dy"], p["x"], t, *w, p["dx_base"])
    for bad in (dict(dA=p["A"]), dict(dB=p["B"]), dict(dB=p["A"].view(L, N, R)), dict(dx=p["dy"]),
                dict(dx=p["x"])):
        with pytest.raises(B.SegQuantError, match="INVALID_ARG"):
            B.sq_lora_backward(*args, **bad)
    wide = torch.zeros(M, K + 8, dtype=BF, device="cuda")
    with pytest.raises(B.SegQuantError, match="INVALID_ARG"):
        B.sq_rope_forward(wide[:, :K], torch.zeros(M, dtype=torch.int32, device="cuda"),
                          torch.rand(8, device="cuda"), 16, out=wide[:, 8:])
    assert all(torch.equal(p[k], v) for k, v in keep.items())
