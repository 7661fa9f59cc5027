"""Rotary positions (sq_rope_forward, sq_rope_backward, sq_rope_frequencies)
against the 64-bit formulas."""
import pytest
import torch

from w8a8_gemm_b200 import binding as B

import ops_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

CASES = [  # M, H, D, rot, axis_pairs, top position
    (1, 1, 8, 2, None, 10), (1, 32, 64, 64, None, 10 ** 6), (3, 5, 64, 32, None, 131072),
    (17, 24, 128, 128, [16, 24, 24], 4096), (130, 2, 80, 48, [12, 12], 99), (9, 3, 96, 20, None, 2 ** 31 - 1),
    (500, 7, 40, 40, [20, 0], 1000), (33, 4, 256, 250, [1, 2, 100, 22], 70), (2049, 1, 16, 6, None, 5000),
    (65, 48, 128, 64, [32], 50),
]


def _inputs(M, H, D, rot, pairs, top, dtype, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(M, H * D, generator=g, device="cuda").to(dtype)
    axes = len(pairs) if pairs else 1
    pos = torch.randint(0, top, (M, axes), generator=g, device="cuda").to(torch.int32)
    pos[0] = top - 1
    if M > 2:
        pos[1] = 0
        pos[2] = -(top // 2)
    f, _ = B.sq_rope_frequencies(rot)
    return x, pos, f.cuda()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", [B.SQ_ROPE_INTERLEAVED, B.SQ_ROPE_HALF])
@pytest.mark.parametrize("M,H,D,rot,pairs,top", CASES)
def test_forward_and_backward(M, H, D, rot, pairs, top, layout, dtype):
    x, pos, f = _inputs(M, H, D, rot, pairs, top, dtype, seed=M + rot)
    for call, sign in ((B.sq_rope_forward, 1.0), (B.sq_rope_backward, -1.0)):
        want, bound = ref.rope(x, pos, f, D, layout, pairs, 1.25, sign)
        got = call(x, pos, f, D, layout=layout, axis_pairs=pairs, factor=1.25)
        ref.check(got, want, bound, "out")
        same = x.clone()
        call(same, pos, f, D, same, layout=layout, axis_pairs=pairs, factor=1.25)
        assert torch.equal(same, got)      # in place


@pytest.mark.parametrize("layout", [B.SQ_ROPE_INTERLEAVED, B.SQ_ROPE_HALF])
def test_q_and_k_columns_of_a_qkv_row(layout):
    """The q|k part of [q | k | v] rows, in place: v and the padding stay; into
    another buffer, the columns past `rot` are copied."""
    M, H, D, rot = 70, 6, 64, 48
    x, pos, f = _inputs(M, 2 * H, D, rot, None, 3000, BF, seed=1)
    rows = torch.full((M, 3 * H * D + 8), float("nan"), dtype=BF, device="cuda")
    rows[:, :2 * H * D] = x
    qk = rows[:, :2 * H * D]
    want, bound = ref.rope(x, pos, f, D, layout, None, 1.0, 1.0)
    other = torch.full((M, 2 * H * D + 16), 2.0, dtype=BF, device="cuda")
    B.sq_rope_forward(qk, pos[:, 0].contiguous(), f, D, other[:, :2 * H * D], layout=layout)
    ref.check(other[:, :2 * H * D].contiguous(), want, bound, "out")
    assert (other[:, 2 * H * D:] == 2.0).all()
    B.sq_rope_forward(qk, pos, f, D, qk, layout=layout)
    assert torch.equal(rows[:, :2 * H * D], other[:, :2 * H * D])
    assert torch.isnan(rows[:, 2 * H * D:]).all()


def test_no_rows_and_capture():
    f = B.sq_rope_frequencies(32)[0].cuda()
    e = torch.empty(0, 64, dtype=BF, device="cuda")
    assert B.sq_rope_forward(e, torch.empty(0, 1, dtype=torch.int32, device="cuda"), f,
                             32).shape == (0, 64)
    x, pos, f = _inputs(100, 4, 64, 64, None, 500, BF, seed=7)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = B.sq_rope_forward(x, pos, f, 64)
    pos.copy_(pos + 1)     # the next token's positions, in the captured buffer
    graph.replay()
    assert torch.equal(y, B.sq_rope_forward(x, pos, f, 64))
