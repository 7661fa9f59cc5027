"""The two ways of the operators' calls from torch to the library, compiled
(csrc/torch_calls.cpp) and through ctypes: the same bits, the same refusals."""
import pytest
import torch

from w8a8_gemm_b200 import binding as B

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _rand(*shape, dtype=BF, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + sum(shape))
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _calls():
    """name -> call of every operator, with and without the optional arguments."""
    M, K, N, R, L = 37, 64, 96, 16, 3
    x, A, Bm = _rand(M, K), _rand(L, R, K), _rand(L, N, R)
    scale, base, dy = _rand(L, dtype=F32), _rand(M, N), _rand(M, N, seed=1)
    ids = torch.arange(M, device="cuda", dtype=torch.int32) % (L + 1) - 1
    plan = B.sq_lora_plan(ids, L)
    t = torch.zeros(M, R, device="cuda")
    B.sq_lora_forward(x, A, Bm, scale, plan, None, t=t)
    wide = _rand(M, 200)
    pos = torch.arange(2 * M, device="cuda", dtype=torch.int32)
    inv = torch.rand(16, device="cuda")
    h, gamma, beta = _rand(2, 50, 64), _rand(64), _rand(64, seed=2)
    mean, rstd = B.sq_group_norm_forward(h, 4, gamma, beta)[1:]
    seg = B.Segments(B.SQ_SEG_INPUT, [0, 32, 64], 1)
    wq = _rand(N, K).mul(30).to(torch.int8)
    s_w, d = torch.rand(2, N, device="cuda"), torch.rand(1, K, device="cuda") + 0.5
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    lf, lb = B.sq_lora_forward, B.sq_lora_backward
    gf, gb, ig = (B.sq_group_norm_forward, B.sq_group_norm_backward,
                  B.sq_dualscale_seglinear_input_grad)
    one = x[:1, :32]
    return {
        "lora": lambda: lf(x, A, Bm, scale, plan, base),
        "lora none": lambda: lf(x, A, Bm, scale, plan, None, t=t.clone(), workspace=ws),
        "lora fp32": lambda: lf(x, A, Bm, scale, plan, base.float(), y=torch.empty(M, N, device="cuda")),
        "lora bwd": lambda: lb(dy, x, t, A, Bm, scale, plan, x),
        "lora bwd fp32": lambda: lb(dy, x, t, A, Bm, scale, plan, None, grad_dtype=F32, workspace=ws),
        "lora bwd no dx": lambda: lb(dy, x, t, A, Bm, scale, plan, None, need_dx=False),
        "lora bwd no weights": lambda: lb(dy, x, t, A, Bm, scale, plan, None, need_weights=False),
        "rope": lambda: B.sq_rope_forward(wide[:, 64:192], pos[:M], inv, 64),
        "rope axes": lambda: B.sq_rope_backward(wide[:, :128], pos.view(M, 2), inv, 32,
                                                layout=B.SQ_ROPE_HALF, axis_pairs=[6, 10],
                                                factor=1.5),
        "rope one": lambda: B.sq_rope_forward(one, pos[:1], inv, 32, out=one.clone()),
        "norm": lambda: gf(h, 4, gamma, beta, act=B.SQ_ACT_GELU),
        "norm bare": lambda: gf(h, 8, None, None, eps=1e-3, workspace=ws),
        "norm bwd": lambda: gb(h, h, 4, gamma, beta, mean, rstd, act=B.SQ_ACT_SILU),
        "norm bwd fp32": lambda: gb(h, h, 4, None, beta, mean, rstd, grad_dtype=F32, need_dx=False),
        "grad": lambda: ig(dy, wq, s_w, d, seg),
        "grad bare": lambda: ig(dy, wq, s_w, None, seg, dx=torch.empty(M, K, dtype=BF, device="cuda")),
        # refusals: the library's, and arguments that do not fit
        "R": lambda: lf(x, A[:, :12].contiguous(), Bm[:, :, :12].contiguous(), scale, plan, base),
        "scale": lambda: lf(x, A, Bm, scale[:2], plan, base),
        "y type": lambda: lf(x, A, Bm, scale, plan, base, y=torch.empty(M, N, device="cuda")),
        "dx unused": lambda: lb(dy, x, t, A, Bm, scale, plan, x, need_dx=False),
        "grad_dtype": lambda: lb(dy, x, t, A, Bm, scale, plan, None, grad_dtype=torch.half),
        "heads": lambda: B.sq_rope_forward(x, pos[:M], inv, 48),
        "axis pairs": lambda: B.sq_rope_forward(x, pos.view(M, 2), inv, 64, axis_pairs=[4, 4]),
        "groups": lambda: gf(h, 5, gamma, beta),
        "no groups": lambda: gf(h, 0, gamma, beta),
        "stride": lambda: gf(h.transpose(0, 1), 4, gamma, beta),
        "eps": lambda: gf(h, 4, gamma, beta, eps=float("nan")),
        "mean": lambda: gb(h, h, 4, gamma, beta, mean[:1], rstd),
        "steps": lambda: ig(dy, wq, s_w[:1], None, seg),
        "workspace": lambda: ig(dy, wq, s_w, None, seg, workspace=ws[:64]),
        "workspace type": lambda: ig(dy, wq, s_w, None, seg, workspace=t),
        "cpu": lambda: ig(dy, wq.cpu(), s_w, None, seg),
        "none": lambda: ig(None, wq, s_w, None, seg),
    }


def _outcome(f):
    try:
        r = f()
    except (ValueError, B.SegQuantError) as e:
        return type(e), str(e)
    return [None if v is None else v.clone() for v in (r if isinstance(r, tuple) else (r,))]


def test_both_ways_agree(monkeypatch):
    calls = _calls()
    assert B._calls(), "csrc/torch_calls.cpp is not built"
    got = {name: _outcome(f) for name, f in calls.items()}
    monkeypatch.setattr(B, "_native", False)
    for name, f in calls.items():
        want = _outcome(f)
        if isinstance(want, tuple):
            assert got[name] == want, name
            continue
        assert len(want) == len(got[name]), name
        for a, b in zip(got[name], want):
            assert (a is None) == (b is None), name
            if a is not None:
                assert a.dtype == b.dtype and a.shape == b.shape, name
                # rows without an adapter leave t as it was: compare what is written
                if name.startswith("lora") and "bwd" not in name and a is got[name][1]:
                    rows = torch.arange(a.shape[0], device="cuda") % 4 != 0
                    a, b = a[rows], b[rows]
                assert torch.equal(a, b), name
    refused = [n for n, v in got.items() if isinstance(v, tuple)]
    assert len(refused) == 17, refused
    assert B.sq_get_device_status() == B.SQ_OK


def test_outputs_are_fresh_and_on_the_callers_stream():
    """A call on a side stream takes its memory and its place there."""
    x, pos = _rand(300, 128), torch.arange(300, device="cuda", dtype=torch.int32)
    inv = torch.rand(32, device="cuda")
    want = B.sq_rope_forward(x, pos, inv, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = B.sq_rope_forward(x, pos, inv, 64)
        b = B.sq_rope_forward(x, pos, inv, 64)
    side.synchronize()
    assert a.data_ptr() != b.data_ptr() and torch.equal(a, want) and torch.equal(b, want)
