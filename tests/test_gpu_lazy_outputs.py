"""Outputs and workspaces that share their storage with another tensor until the
first write (copy on write): the other tensor keeps its values."""
import pytest
import torch

from w8a8_gemm_b200 import binding as B

from test_gpu_lora import _problem

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _calls():
    """name -> (call with one output given, shape and type of that output)."""
    M, K, N, R, L = 50, 64, 72, 8, 2
    p = _problem(M, K, N, R, L, seed=2, spread="one")
    w = (p["A"], p["B"], p["scale"], B.sq_lora_plan(p["ids"], L))
    t = B.sq_lora_forward(p["x"], *w, None)[1]
    pos, inv = torch.arange(M, dtype=torch.int32, device="cuda"), torch.rand(16, device="cuda")
    h = p["x"].view(2, 25, K)
    mean, rstd = B.sq_group_norm_forward(h, 4, None, None)[1:]
    wq, s_w = torch.ones(N, K, dtype=torch.int8, device="cuda"), torch.ones(1, N, device="cuda")
    back = (p["dy"], p["x"], t, *w)

    def grad(**k):
        return B.sq_dualscale_seglinear_input_grad(p["dy"], wq, s_w, None, B.Segments(), **k)

    return {
        "lora y": (lambda o: B.sq_lora_forward(p["x"], *w, p["base"], y=o), (M, N), BF),
        "lora y in place": (lambda o: B.sq_lora_forward(p["x"], *w, o, y=o), (M, N), BF),
        "lora t": (lambda o: B.sq_lora_forward(p["x"], *w, p["base"], t=o), (M, R), F32),
        "lora dx": (lambda o: B.sq_lora_backward(*back, None, dx=o), (M, K), BF),
        "lora dx in place": (lambda o: B.sq_lora_backward(*back, o, dx=o), (M, K), BF),
        "lora dA": (lambda o: B.sq_lora_backward(*back, None, dA=o), (L, R, K), BF),
        "lora dB": (lambda o: B.sq_lora_backward(*back, None, dB=o), (L, N, R), BF),
        "rope": (lambda o: B.sq_rope_forward(p["x"], pos, inv, 32, out=o), (M, K), BF),
        "rope in place": (lambda o: B.sq_rope_forward(o, pos, inv, 32, out=o), (M, K), BF),
        "norm y": (lambda o: B.sq_group_norm_forward(h, 4, None, None, y=o), (2, 25, K), BF),
        "norm dx": (lambda o: B.sq_group_norm_backward(h, h, 4, None, None, mean, rstd, dx=o),
                    (2, 25, K), BF),
        "grad dx": (lambda o: grad(dx=o), (M, K), BF),
        "grad workspace": (lambda o: grad(workspace=o),
                           (B.sq_input_grad_workspace_bytes(N, K),), torch.uint8),
    }


@pytest.mark.parametrize("native", [True, False])
def test_the_original_keeps_its_values(native, monkeypatch):
    if not native:
        monkeypatch.setattr(B, "_native", False)
    wrong = []
    for name, (call, shape, dtype) in _calls().items():
        original = torch.full(shape, 1, dtype=dtype, device="cuda")
        lazy, plain = torch._lazy_clone(original), original.clone()
        first = call(lazy)
        want = call(plain)
        if not (original == 1).all():
            wrong.append(f"{name}: written through")
        elif name != "grad workspace" and not torch.equal(lazy, plain):
            wrong.append(f"{name}: differs")
        del first, want
    assert not wrong, wrong


def test_lazy_inputs_are_read_and_stay_lazy():
    M, K, N, R, L = 50, 64, 72, 8, 2
    p = _problem(M, K, N, R, L, seed=2, spread="one")
    plan = B.sq_lora_plan(p["ids"], L)
    x = torch._lazy_clone(p["x"])
    want = B.sq_lora_forward(p["x"], p["A"], p["B"], p["scale"], plan, p["base"])[0]
    assert torch.equal(want, B.sq_lora_forward(x, p["A"], p["B"], p["scale"], plan, p["base"])[0])
