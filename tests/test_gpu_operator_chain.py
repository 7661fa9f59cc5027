"""The operators as they are used together: group norm, quantized q|k|v
projection with adapters, rotary positions, and back (layer.AttentionInput).
Values and gradients against 64 bits with bounds that are carried through the
chain; the same bits from a side stream and from replayed graphs."""
import pytest
import torch

from w8a8_gemm_b200 import binding as B
from w8a8_gemm_b200.layer import Adapters, AttentionInput, DualScaleSegLinear

import ops_ref as ref

pytestmark = pytest.mark.gpu
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64

CASES = [  # B, S, C, groups, heads of q and of k|v, head_dim, rot, L, R, layer
    dict(B=1, S=1, C=64, groups=0, hq=2, hk=1, D=16, rot=16, L=3, R=8, kind="plain"),
    dict(B=2, S=77, C=320, groups=32, hq=4, hk=4, D=40, rot=24, L=4, R=16, kind="plain"),
    dict(B=1, S=300, C=256, groups=8, hq=8, hk=2, D=64, rot=64, L=2, R=72, kind="divisor"),
    dict(B=3, S=50, C=128, groups=16, hq=2, hk=2, D=32, rot=32, L=5, R=8, kind="w4"),
    dict(B=1, S=130, C=192, groups=4, hq=3, hk=1, D=64, rot=32, L=1, R=32, kind="fp8"),
]


def _make(B_, S, C, groups, hq, hk, D, rot, L, R, kind, seed=5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + C)

    def rand(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF)

    N = (hq + 2 * hk) * D
    x = rand(B_, S, C)
    w, bias = rand(N, C, scale=C ** -0.5), rand(N, scale=0.1)
    d = torch.exp(0.3 * torch.randn(1, C, generator=g, device="cuda")) if kind == "divisor" else None
    seg = B.Segments(B.SQ_SEG_NONE)
    layer = DualScaleSegLinear(w, bias, d, seg, rand(256, C), weight_bits=4 if kind == "w4" else 8,
                               fp8=kind == "fp8")
    ad = Adapters(rand(L, R, C, scale=C ** -0.5), rand(L, N, R, scale=R ** -0.5),
                  torch.rand(L, generator=g, device="cuda") + 0.5)
    inv, factor = B.sq_rope_frequencies(rot)
    axes = [rot // 4, rot // 2 - rot // 4]
    pos = torch.randint(0, 512, (B_ * S, 2), generator=g, device="cuda", dtype=torch.int32)
    ids = torch.randint(-1, L, (B_ * S,), generator=g, device="cuda", dtype=torch.int32)
    norm = dict(groups=groups, gamma=(1 + rand(C, scale=0.1).float()).to(BF),
                beta=rand(C, scale=0.1), act=B.SQ_ACT_SILU) if groups else {}
    front = AttentionInput(layer, D, hq + hk, inv.cuda(), factor, layout=B.SQ_ROPE_HALF,
                           axis_pairs=axes, **norm)
    return front, ad, x, pos, ids, rand(B_ * S, N)


def _weights(layer):
    """W~ of the layer in 64 bits."""
    if layer.fp8:
        codes = layer.wq.view(torch.float8_e4m3fn).double()
    elif layer.wq4 is not None:
        B.sq_unpack_weight_w4(layer.wq4, layer.wq)
        codes = layer.wq.double() / 16
    else:
        codes = layer.wq.double()
    return ref.dequantized(codes, layer.s_w, layer.d, 0, None, 1)


def _rounded(v, e):
    return e + ref.U[BF] * (v.abs() + e)


def _gn_error(e, x, G, gamma, beta, mean, rstd, kind):
    """What an error of at most e in dy makes of dx, dgamma and dbeta, which are
    linear in dy: every term by its magnitude."""
    B_, S, C = x.shape
    n = S * C // G
    mu, rs = ref._per_channel(mean, C), ref._per_channel(rstd, C)
    xh = (x.to(F64) - mu) * rs
    dv = e * ref.act(xh * gamma.to(F64) + beta.to(F64), kind)[1].abs()
    h = dv * gamma.to(F64).abs()

    def mean_of(t):
        return ref._per_channel(t.reshape(B_, S, G, C // G).sum((1, 3)) / n, C)

    return {"dx": rs * (h + mean_of(h) + xh.abs() * mean_of(h * xh.abs())),
            "dgamma": (dv * xh.abs()).sum((0, 1)), "dbeta": dv.sum((0, 1))}


def _turn(front, v, e, pos, sign):
    """The rotary columns of v turned, with errors e: |cos| and |sin| are at most 1."""
    n, D, pairs = front.turned, front.head_dim, front.inv_freq.numel()
    r, er = ref.rope(v[:, :n], pos, front.inv_freq, D, 1, front.axis_pairs, front.factor, sign)
    z = e[:, :n].reshape(len(e), -1, D).clone()
    both = abs(front.factor) * (z[..., :pairs] + z[..., pairs:2 * pairs])
    z[..., :pairs] = both
    z[..., pairs:2 * pairs] = both
    w, ew = v.clone(), e.clone()
    w[:, :n], ew[:, :n] = r, z.reshape(len(e), -1) + er
    return w, ew


def _carried(eg, h, t, ad, ids):
    """What an error eg of the projection's output gradient makes of dA, dB, dx."""
    e = {"dA": torch.zeros(ad.A.shape, dtype=F64, device="cuda"),
         "dB": torch.zeros(ad.B.shape, dtype=F64, device="cuda"),
         "dx": torch.zeros(h.shape, dtype=F64, device="cuda")}
    for a in range(ad.A.shape[0]):
        r = (ids == a).nonzero()[:, 0]
        edt = float(ad.scale[a]) * (eg[r] @ ad.B[a].to(F64).abs())
        e["dB"][a] = float(ad.scale[a]) * (eg[r].t() @ t[r].to(F64).abs())
        e["dA"][a] = edt.t() @ h[r].to(F64).abs()
        e["dx"][r] = edt @ ad.A[a].to(F64).abs()
    return e


@pytest.mark.parametrize("case", CASES, ids=lambda c: c["kind"] + str(c["S"]))
def test_values_and_gradients(case):
    c = dict(case)
    front, ad, x, pos, ids, dy = _make(c.pop("B"), **c)
    layer, C, turned = front.qkv, case["C"], front.turned
    out, saved = front(x, pos, ad, ad.plan(ids))
    h = saved[1]
    if front.groups:
        want, wm, wr = ref.group_norm_forward(x, front.groups, front.gamma, front.beta, front.eps,
                                              front.act)
        ref.check(h.view(x.shape), *want, "h")
    base = layer(h)   # the projection itself is pinned to the oracle elsewhere
    y, ey, t, et = ref.lora_forward(h, ad.A, ad.B, ad.scale, ids, base, BF)
    ey = _rounded(y, ey)
    ref.check(out, *_turn(front, y, ey, pos, 1.0), "q|k|v")
    # backward: the gradient g of the projection's output, dx and the parameters
    grads = front.backward(dy.clone(), saved, grad_dtype=F32)
    g, eg = _turn(front, dy.to(F64), torch.zeros(dy.shape, dtype=F64, device="cuda"), pos, -1.0)
    eg[:, :turned] = _rounded(g, eg)[:, :turned]
    W = _weights(layer)
    b, eb = ref.input_grad(g, W)
    eb = _rounded(b, eb + eg @ W.abs())
    want = ref.lora_backward(g, h, saved[4], ad.A, ad.B, ad.scale, ids, b, F32)
    ea = _carried(eg, h, saved[4], ad, ids)
    ea["dx"] += eb
    ref.check(grads.A, want["dA"][0], want["dA"][1] + ea["dA"], "dA")
    ref.check(grads.B, want["dB"][0], want["dB"][1] + ea["dB"], "dB")
    v, e = want["dx"][0], want["dx"][1] + ea["dx"]
    if not front.groups:
        ref.check(grads.x.view(-1, C), v, e, "dx")
        assert grads.gamma is None and grads.beta is None
        return
    v, e = v.view(x.shape), _rounded(v, e).view(x.shape)
    norm = (x, front.groups, front.gamma, front.beta, saved[2], saved[3], front.act)
    want = ref.group_norm_backward(v, *norm)
    carried = _gn_error(e, *norm)
    for name, got in (("dx", grads.x), ("dgamma", grads.gamma), ("dbeta", grads.beta)):
        ref.check(got, want[name][0], want[name][1] + carried[name], name)


def test_without_adapters_and_the_layers_own_calls():
    """No adapters: the projection alone; all rows without one: the same bits."""
    c = dict(CASES[1])
    front, ad, x, pos, ids, dy = _make(c.pop("B"), **c)
    plain, saved = front(x, pos)
    none, saved_none = front(x, pos, ad, ad.plan(torch.full_like(ids, -1)))
    assert torch.equal(plain, none)
    a, b = front.backward(dy.clone(), saved), front.backward(dy.clone(), saved_none)
    assert a.A is None and a.B is None and torch.equal(a.x, b.x) and torch.equal(a.gamma, b.gamma)
    assert not b.A.any() and not b.B.any()
    with pytest.raises(ValueError):
        front(x, pos, ad)


def test_differences_of_the_adapters():
    """The loss <out, dy> along a direction of A and of B, that in which it grows.
    With A or B moved alone it is linear in the move, so the difference quotient
    is the derivative but for the errors of the two ends and of the gradient,
    each within its bound of the tests above."""
    c = dict(CASES[2])
    front, ad, x, pos, ids, dy = _make(c.pop("B"), **c)
    plan = ad.plan(ids)
    out, saved = front(x, pos, ad, plan)
    h, t = saved[1], saved[4]
    base = front.qkv(h)
    grads = front.backward(dy.clone(), saved, grad_dtype=F32)
    g, eg = _turn(front, dy.to(F64), torch.zeros(dy.shape, dtype=F64, device="cuda"), pos, -1.0)
    eg[:, :front.turned] = _rounded(g, eg)[:, :front.turned]
    want = ref.lora_backward(g, h, t, ad.A, ad.B, ad.scale, ids, None, F32)
    carried = _carried(eg, h, t, ad, ids)
    weight = dy.to(F64).abs()
    for name in ("A", "B"):
        at, grad = getattr(ad, name), getattr(grads, name)
        ends, allowed = [], 0.0
        for s in (1, -1):
            moved = Adapters(ad.A, ad.B, ad.scale)
            setattr(moved, name, (at + s * 2 * at.abs() * grad.sign()).to(BF))
            got = front(x, pos, moved, plan)[0].to(F64)
            y, ey, _, _ = ref.lora_forward(h, moved.A, moved.B, moved.scale, ids, base, BF)
            v, e = _turn(front, y, _rounded(y, ey), pos, 1.0)
            allowed += float((_rounded(v, e) * weight).sum())
            ends.append((getattr(moved, name).to(F64), got))
        used = ends[0][0] - ends[1][0]
        quotient = float(((ends[0][1] - ends[1][1]) * dy.to(F64)).sum())
        slope = float((grad.to(F64) * used).sum())
        v, e = want["d" + name]
        e = e + carried["d" + name]
        allowed += float(((e + ref.U[F32] * (v.abs() + e)) * used.abs()).sum())
        assert abs(quotient - slope) <= allowed, (name, quotient, slope, allowed)


def test_side_stream_and_two_replayed_graphs():
    """The chain on another stream, and captured twice (forward and backward in
    each graph, the two graphs replayed in turn): the same bits every time."""
    c = dict(CASES[1])
    front, ad, x, pos, ids, dy = _make(c.pop("B"), **c)
    plan = ad.plan(ids)

    def run():
        out, saved = front(x, pos, ad, plan)
        gr = front.backward(dy.clone(), saved)
        return [out, gr.x, gr.A, gr.B, gr.gamma, gr.beta]

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = run()
        graphs.append((graph, res))
    for _ in range(3):
        for graph, res in graphs:
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, res))
    assert B.sq_get_device_status() == B.SQ_OK


def test_empty_batch_and_a_slice_of_wider_features():
    c = dict(CASES[1])
    front, ad, x, pos, ids, dy = _make(c.pop("B"), **c)
    for a in (None, ad):
        out, saved = front(x[:0], pos[:0], a, None if a is None else a.plan(ids[:0]))
        g = front.backward(dy[:0].clone(), saved)
        assert out.shape == (0, front.qkv.N) and g.x.shape == x[:0].shape
        assert not g.gamma.any() and not g.beta.any()
        assert (g.A is None) if a is None else not (g.A.any() or g.B.any())
    C = x.shape[2]
    wide = torch.full((*x.shape[:2], C + 80), float("nan"), dtype=BF, device="cuda")
    part = wide[:, :, 40:40 + C]
    part.copy_(x)
    plan = ad.plan(ids)
    want, got = front(x, pos, ad, plan), front(part, pos, ad, plan)
    assert torch.equal(want[0], got[0])
    a, b = front.backward(dy.clone(), want[1]), front.backward(dy.clone(), got[1])
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    assert B.sq_get_device_status() == B.SQ_OK


def test_host_threads_on_streams_of_their_own():
    """Four threads make the same calls at once, each on its stream."""
    import threading
    c = dict(CASES[1])
    front, ad, x, pos, ids, dy = _make(c.pop("B"), **c)
    plan, rows, layer = ad.plan(ids), x.view(-1, x.shape[2]), front.qkv
    torch.cuda.synchronize()
    results = {}

    def run(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(30):
                y, t = B.sq_lora_forward(rows, ad.A, ad.B, ad.scale, plan, None)
                grads = B.sq_lora_backward(dy, rows, t, ad.A, ad.B, ad.scale, plan, None)
                h = B.sq_group_norm_forward(x, 32, front.gamma, front.beta, act=front.act)
                g = B.sq_group_norm_backward(x, x, 32, front.gamma, front.beta, *h[1:])
                d = B.sq_dualscale_seglinear_input_grad(dy, layer.wq, layer.s_w, None, layer.seg)
                q = B.sq_rope_forward(dy, pos, front.inv_freq, front.head_dim,
                                      axis_pairs=front.axis_pairs)
        stream.synchronize()
        results[i] = [y, *grads, *h, *g, d, q]

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert len(results) == 4
    for i in range(1, 4):
        assert all(torch.equal(a, b) for a, b in zip(results[0], results[i]))
    assert B.sq_get_device_status() == B.SQ_OK
