"""The input gradient of a frozen quantized linear
(sq_dualscale_seglinear_input_grad) against the 64-bit product."""
import pytest
import torch

from w8a8_gemm_b200 import binding as B

import ops_ref as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

CASES = [  # M, N, K, mode, segments, groups, divisor
    (1, 16, 16, B.SQ_SEG_NONE, 1, 1, False), (1, 1536, 1536, B.SQ_SEG_INPUT, 24, 1, True),
    (77, 100, 48, B.SQ_SEG_NONE, 1, 1, True), (129, 1, 64, B.SQ_SEG_NONE, 1, 1, False),
    (200, 384, 272, B.SQ_SEG_OUTPUT, 3, 3, True), (300, 768, 1024, B.SQ_SEG_OUTPUT, 6, 1, True),
    (1000, 515, 1600, B.SQ_SEG_NONE, 1, 1, False), (2048, 640, 2304, B.SQ_SEG_INPUT, 6, 1, False),
    (5000, 72, 1040, B.SQ_SEG_NONE, 1, 1, True),
]


def _layer(N, K, mode, n, G, divisor, flags, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    extent = {B.SQ_SEG_NONE: 1, B.SQ_SEG_INPUT: K, B.SQ_SEG_OUTPUT: N}[mode]
    off = None if mode == B.SQ_SEG_NONE else [extent * i // n for i in range(n + 1)]
    seg = B.Segments(mode, off, G, flags)
    wq = torch.randint(-128, 128, (N, K), generator=g, device="cuda").to(torch.int8)
    s_w = torch.rand(seg.S, N, generator=g, device="cuda") * 0.01 + 1e-4
    d = torch.exp(torch.randn(G, K, generator=g, device="cuda")) if divisor else None
    return seg, wq, s_w, d, g


def _codes(wq, flags):
    if flags & B.SQ_FLAG_FP8:
        return wq.view(torch.float8_e4m3fn).double()
    return wq.double() / (16 if flags & B.SQ_FLAG_W4 else 1)


@pytest.mark.parametrize("M,N,K,mode,n,G,divisor", CASES)
@pytest.mark.parametrize("flags", [0, B.SQ_FLAG_W4, B.SQ_FLAG_FP8, B.SQ_FLAG_SINGLE_SCALE])
def test_input_grad(M, N, K, mode, n, G, divisor, flags):
    seg, wq, s_w, d, g = _layer(N, K, mode, n, G, divisor, flags, seed=M + N)
    if flags & B.SQ_FLAG_FP8:      # no NaN codes: 0x7F and 0xFF are never made
        wq = torch.where((wq & 0x7F) == 0x7F, torch.zeros_like(wq), wq)
    ld = (N + 7) // 8 * 8
    rows = torch.full((M, ld + 8), float("nan"), dtype=BF, device="cuda")
    dy = rows[:, :N]
    dy.copy_(torch.randn(M, N, generator=g, device="cuda"))
    out = torch.full((M, K + 8), 4.0, dtype=BF, device="cuda")
    B.sq_dualscale_seglinear_input_grad(dy, wq, s_w, d, seg, dx=out[:, :K])
    w = ref.dequantized(_codes(wq, flags), s_w, d, mode, seg.offsets, G)
    ref.check(out[:, :K].contiguous(), *ref.input_grad(dy, w), "dx")
    assert (out[:, K:] == 4.0).all()
    assert B.sq_get_device_status() == B.SQ_OK


def test_no_rows_capture_and_a_shared_workspace():
    """Two layers share one workspace on a stream; a replayed graph gives the
    same bits."""
    seg, wq, s_w, d, g = _layer(256, 320, B.SQ_SEG_NONE, 1, 1, True, 0, seed=1)
    seg2, wq2, s_w2, d2, _ = _layer(128, 192, B.SQ_SEG_INPUT, 3, 1, True, 0, seed=2)
    e = B.sq_dualscale_seglinear_input_grad(torch.empty(0, 256, dtype=BF, device="cuda"), wq, s_w,
                                            d, seg)
    assert e.shape == (0, 320)
    dy = torch.randn(500, 256, generator=g, device="cuda").to(BF)
    dy2 = torch.randn(70, 128, generator=g, device="cuda").to(BF)
    one = B.sq_dualscale_seglinear_input_grad(dy, wq, s_w, d, seg)
    two = B.sq_dualscale_seglinear_input_grad(dy2, wq2, s_w2, d2, seg2)
    ws = torch.empty(B.sq_input_grad_workspace_bytes(256, 320), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = B.sq_dualscale_seglinear_input_grad(dy, wq, s_w, d, seg, workspace=ws)
        b = B.sq_dualscale_seglinear_input_grad(dy2, wq2, s_w2, d2, seg2, workspace=ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, one) and torch.equal(b, two)


@pytest.mark.parametrize("M,N,K,mode,n,G,divisor", [
    (1, 1536, 128, B.SQ_SEG_NONE, 1, 1, True), (256, 1500, 1920, B.SQ_SEG_INPUT, 4, 1, False),
    (257, 1536, 896, B.SQ_SEG_OUTPUT, 4, 4, True), (200, 6000, 16, B.SQ_SEG_NONE, 1, 1, False),
    (700, 2000, 656, B.SQ_SEG_NONE, 1, 1, True), (1025, 1600, 768, B.SQ_SEG_INPUT, 6, 1, False),
    (3, 4095, 1808, B.SQ_SEG_NONE, 1, 1, True)])
def test_long_contractions_of_few_tiles(M, N, K, mode, n, G, divisor):
    """Several pairs of blocks share a tile's contraction: values, the rows and
    columns past the last left alone, the same bits from a replayed graph."""
    seg, wq, s_w, d, g = _layer(N, K, mode, n, G, divisor, 0, seed=N)
    ld = (N + 7) // 8 * 8
    dy = torch.full((M, ld + 8), float("nan"), dtype=BF, device="cuda")[:, :N]
    dy.copy_(torch.randn(M, N, generator=g, device="cuda"))
    out = torch.full((M + 2, K + 8), 4.0, dtype=BF, device="cuda")
    B.sq_dualscale_seglinear_input_grad(dy, wq, s_w, d, seg, dx=out[:M, :K])
    w = ref.dequantized(_codes(wq, 0), s_w, d, mode, seg.offsets, G)
    ref.check(out[:M, :K].contiguous(), *ref.input_grad(dy, w), "dx")
    assert (out[:, K:] == 4.0).all() and (out[M:] == 4.0).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = B.sq_dualscale_seglinear_input_grad(dy, wq, s_w, d, seg)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, out[:M, :K])
    assert B.sq_get_device_status() == B.SQ_OK
