"""A single row's stride says nothing: rows cut from buffers of any width."""
import pytest
import torch

from w8a8_gemm_b200 import binding as B

from test_gpu_lora import _problem

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _cut(t, stride):
    """t [1, n] with another row stride, which no element uses."""
    return torch.as_strided(t, t.shape, (stride, 1))


@pytest.mark.parametrize("native", [True, False])
@pytest.mark.parametrize("extra", [0, 1, 3, 4, 12])
def test_a_row_of_a_buffer_of_any_width(extra, native, monkeypatch):
    if not native:
        monkeypatch.setattr(B, "_native", False)
    K, N, R, L = 64, 80, 8, 2
    p = _problem(1, K, N, R, L, seed=8, spread="one")
    far = {k: _cut(p[k], p[k].shape[1] + extra) for k in ("x", "base", "dy", "dx_base")}
    plan = B.sq_lora_plan(p["ids"], L)
    w = (p["A"], p["B"], p["scale"], plan)
    y, t = B.sq_lora_forward(p["x"], *w, p["base"])
    z, _ = B.sq_lora_forward(far["x"], *w, far["base"])
    assert torch.equal(y, z)
    here = _cut(p["base"].clone(), N + extra)
    B.sq_lora_forward(far["x"], *w, here, y=here)
    assert torch.equal(y, here)
    want = B.sq_lora_backward(p["dy"], p["x"], t, *w, p["dx_base"])
    got = B.sq_lora_backward(far["dy"], far["x"], t, *w, far["dx_base"])
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    pos = torch.tensor([17], dtype=torch.int32, device="cuda")
    inv = torch.rand(8, device="cuda")
    assert torch.equal(B.sq_rope_forward(p["x"], pos, inv, 16),
                       B.sq_rope_forward(far["x"], pos, inv, 16))
    wq = torch.ones(N, K, dtype=torch.int8, device="cuda")
    s_w = torch.ones(1, N, device="cuda")
    assert torch.equal(B.sq_dualscale_seglinear_input_grad(p["dy"], wq, s_w, None, B.Segments()),
                       B.sq_dualscale_seglinear_input_grad(far["dy"], wq, s_w, None, B.Segments()))
