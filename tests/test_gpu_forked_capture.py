"""The operators captured behind other work than kernels of their own stream: a
copy, a memset, and a join with a side stream whose kernels make the inputs; two
graphs replayed in turn."""
import pytest
import torch

from w8a8_gemm_b200 import binding as B

from test_gpu_lora import _problem

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("M,L", [(12, 2), (700, 3)])
def test_capture_behind_copies_memsets_and_joins(M, L):
    K, N, R = 128, 256, 16
    p = _problem(M, K, N, R, L, seed=M, spread="scattered")
    w = (p["A"], p["B"], p["scale"])
    plan = B.sq_lora_plan(p["ids"], L)
    pos, inv = torch.arange(M, dtype=torch.int32, device="cuda"), torch.rand(16, device="cuda")
    wq, s_w = torch.ones(N, K, dtype=torch.int8, device="cuda"), torch.rand(1, N, device="cuda")
    sources = [p["x"], p["x"].flip(0).contiguous()]

    def chain(x, y, dy):
        h, mean, rstd = B.sq_group_norm_forward(x.view(1, M, K), 4, None, None, act=B.SQ_ACT_SILU)
        B.sq_lora_forward(h.view(M, K), *w, plan, y, y=y)
        B.sq_rope_forward(y[:, :128], pos, inv, 32, out=y[:, :128])
        return y.clone(), B.sq_dualscale_seglinear_input_grad(dy, wq, s_w, None, B.Segments())

    def build(x, src, y, dy, side):
        main = torch.cuda.current_stream()
        x.copy_(src)                                    # a copy ahead of the first kernel
        y.zero_()
        side.wait_stream(main)
        with torch.cuda.stream(side):                   # kernels of another stream
            dy.copy_(p["dy"] * 2)
            other = B.sq_rope_forward(x, pos, inv, 32)
        out = chain(x, y, p["dy"])
        main.wait_stream(side)                          # joined: the next kernel has two ahead
        more = B.sq_lora_backward(dy, x, torch.ones(M, R, device="cuda"), *w, plan, None)
        return (*out, other, *more)

    side = torch.cuda.Stream()
    want, graphs = [], []
    for src in sources:
        x, y, dy = torch.empty_like(p["x"]), torch.empty_like(p["base"]), torch.empty_like(p["dy"])
        want.append([v.clone() for v in build(x, src, y, dy, side)])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = build(x, src, y, dy, side)
        graphs.append((graph, got, (x, y, dy)))
    for _ in range(5):
        for graph, _, _ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for (_, got, _), ref in zip(graphs, want):
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert B.sq_get_device_status() == B.SQ_OK
