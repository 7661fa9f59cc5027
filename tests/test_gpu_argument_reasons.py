"""Arguments that are no tensors, and numbers far out of range, are refused with a
reason by both ways of the operators' calls."""
import pytest
import torch

from w8a8_gemm_b200 import binding as B

from test_gpu_lora import _problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("native", [True, False])
def test_no_tensors_and_far_numbers(native, monkeypatch):
    if not native:
        monkeypatch.setattr(B, "_native", False)
    M, K, N, R, L = 20, 64, 72, 8, 2
    p = _problem(M, K, N, R, L, seed=5, spread="one")
    x, w = p["x"], (p["A"], p["B"], p["scale"], B.sq_lora_plan(p["ids"], L))
    pos, inv = torch.zeros(M, dtype=torch.int32, device="cuda"), torch.rand(8, device="cuda")
    h = x.view(1, M, K)
    wq, s_w = torch.ones(N, K, dtype=torch.int8, device="cuda"), torch.ones(1, N, device="cuda")
    for match, call in {
            "base": lambda: B.sq_lora_forward(x, *w, 3.0),
            "y must": lambda: B.sq_lora_forward(x, *w, None, y=[1]),
            "workspace": lambda: B.sq_lora_forward(x, *w, None, workspace="many"),
            "inv_freq is required": lambda: B.sq_rope_forward(x, pos, None, 16),
            "inv_freq must": lambda: B.sq_rope_forward(x, pos, [1.0], 16),
            "positions": lambda: B.sq_rope_forward(x, 7, inv, 16),
            "gamma": lambda: B.sq_group_norm_forward(h, 8, 1.0, None),
            "mean": lambda: B.sq_group_norm_backward(h, h, 8, None, None, None, None),
            "s_w": lambda: B.sq_dualscale_seglinear_input_grad(p["dy"], wq, 1.0, None, B.Segments()),
    }.items():
        with pytest.raises(ValueError, match=match):
            call()
    for groups in (0, -1, K + 1, 10 ** 12, -10 ** 12):
        with pytest.raises(B.SegQuantError, match="INVALID_ARG"):
            B.sq_group_norm_forward(h, groups, None, None)
