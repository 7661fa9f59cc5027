"""Cases of the operators that only the bounds-checked debug build runs
(tests/test_gpu_operators_bounds.py starts them in a child process): a plan with a
row past the batch's last.  The buffers really have more rows, so that every
access lies in its allocation; the kernels are told of the first M alone."""
import pytest
import torch

from w8a8_gemm_b200 import binding as B

from test_gpu_lora import _problem

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _doctored(ids, L, place, row):
    """The plan of a batch whose rows all have adapter 0, with `row` at one place."""
    plan = B.sq_lora_plan(ids, L)
    at = (4 + L + 2 + 3) // 4 * 4
    assert plan[at:at + 2].tolist() == [0, min(128, len(ids))]
    plan[at + 3] = 0                  # no neighbours any more
    plan[at + 4 + place] = row
    return plan


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M", [12, 100])      # one kernel for few rows, two kernels
def test_a_row_past_the_batch_is_skipped_and_reported(M, out):
    assert B.sq_debug_bounds_checks()
    K, N, R, L, more = 64, 72, 16, 2, 160
    p = _problem(more, K, N, R, L, seed=1, spread="one", out=out)
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    plan = _doctored(ids, L, M - 1, M + 7)
    y = torch.full((more, N), 9.0, dtype=out, device="cuda")
    t = torch.full((more, R), 9.0, device="cuda")
    w = (p["A"], p["B"], p["scale"])
    B.sq_lora_forward(p["x"][:M], *w, plan, p["base"][:M], y=y[:M], t=t[:M])
    assert B.sq_get_device_status() == B.SQ_ERR_DEVICE_BOUNDS
    assert (y[M - 1:] == 9.0).all() and (t[M - 1:] == 9.0).all()
    good, tg = B.sq_lora_forward(p["x"][:M], *w, B.sq_lora_plan(ids, L), p["base"][:M])
    assert torch.equal(y[:M - 1], good[:M - 1]) and torch.equal(t[:M - 1], tg[:M - 1])
    dx = torch.full((more, K), 9.0, dtype=BF, device="cuda")
    t[M - 1:] = 1.0
    B.sq_lora_backward(p["dy"][:M], p["x"][:M], t[:M], *w, plan, p["dx_base"][:M], dx=dx[:M],
                       need_weights=False)
    assert B.sq_get_device_status() == B.SQ_ERR_DEVICE_BOUNDS
    assert (dx[M - 1:] == 9.0).all()
    assert B.sq_get_device_status() == B.SQ_OK
