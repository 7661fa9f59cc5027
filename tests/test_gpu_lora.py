"""Low-rank adapters beside a shared projection (sq_lora_plan, _forward,
_backward) against the 64-bit formulas, within bounds that count roundings."""
import pytest
import torch

from w8a8_gemm_b200 import binding as B

import ops_ref as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _problem(M, K, N, R, L, seed, spread="runs", out=BF):
    g = _gen(seed)

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda")

    x = (randn(M, K) * torch.exp(randn(K))).to(BF)
    A = (randn(L, R, K) * K ** -0.5).to(BF)
    Bm = (randn(L, N, R) * 0.2).to(BF)
    scale = torch.rand(L, generator=g, device="cuda") * 2 - 0.5
    if spread == "runs":       # ragged neighbouring requests, some without an adapter
        cuts = torch.sort(torch.randint(0, M + 1, (max(1, min(M, 6)),), generator=g,
                                        device="cuda")).values
        req = torch.searchsorted(cuts, torch.arange(M, device="cuda"), right=True)
        ids = torch.randint(-1, L, (len(cuts) + 1,), generator=g, device="cuda")[req]
    elif spread == "scattered":  # any row any adapter
        ids = torch.randint(-1, L, (M,), generator=g, device="cuda")
    elif spread == "mixed":    # long runs, and between them rows of any adapter
        ids = (torch.arange(M, device="cuda") // 700) % (L + 1) - 1
        loose = torch.rand(M, generator=g, device="cuda") < 0.3
        ids = torch.where(loose & (torch.arange(M, device="cuda") % 1500 < 600),
                          torch.randint(-1, L, (M,), generator=g, device="cuda"), ids)
    elif spread == "one":
        ids = torch.full((M,), L - 1, device="cuda")
    else:                      # no row has one; numbers out of range mean none, too
        ids = torch.full((M,), -1, device="cuda")
        ids[::3] = L + 5
        ids[1::3] = -2 ** 31
    base = randn(M, N).to(out)
    dy = randn(M, N).to(BF)
    return dict(x=x, A=A, B=Bm, scale=scale, ids=ids.to(torch.int32), base=base, dy=dy,
                dx_base=randn(M, K).to(BF))


SIZES = [  # M, K, N, R, L, spread
    (1, 64, 64, 8, 1, "one"), (1, 1536, 1536, 16, 4, "scattered"), (16, 256, 328, 16, 8, "scattered"),
    (63, 72, 200, 24, 3, "runs"), (64, 8, 8, 8, 2, "scattered"), (65, 128, 136, 32, 2, "one"),
    (333, 1000, 520, 48, 5, "runs"), (130, 2056, 264, 64, 3, "scattered"), (257, 512, 384, 128, 2, "runs"),
    (129, 200, 1160, 96, 7, "scattered"), (1500, 448, 640, 40, 3, "runs"), (77, 64, 128, 16, 40, "scattered"),
    (3000, 320, 3080, 72, 2, "scattered"), (5000, 256, 2048, 64, 3, "mixed"), (100, 64, 72, 8, 3, "none"), (300, 96, 64, 16, 1024, "scattered"), (4100, 256, 256, 64, 1, "one"),
]


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,K,N,R,L,spread", SIZES)
def test_forward(M, K, N, R, L, spread, out):
    p = _problem(M, K, N, R, L, seed=M + R, spread=spread, out=out)
    plan = B.sq_lora_plan(p["ids"], L)
    t = torch.full((M, R), -7.5, device="cuda")
    y, t = B.sq_lora_forward(p["x"], p["A"], p["B"], p["scale"], plan, p["base"], t=t)
    assert y.dtype == out
    yr, ye, tr, te = ref.lora_forward(p["x"], p["A"], p["B"], p["scale"], p["ids"], p["base"], out)
    ref.check(y, yr, ye, "y")
    has = (p["ids"] >= 0) & (p["ids"] < L)
    ref.check(t[has], tr[has], te[has], "t")
    assert (t[~has] == -7.5).all()          # rows without an adapter: t left as it was
    assert torch.equal(y[~has], p["base"][~has])
    assert B.sq_get_device_status() == B.SQ_OK


@pytest.mark.parametrize("grads", [BF, F32])
@pytest.mark.parametrize("M,K,N,R,L,spread", SIZES)
def test_backward(M, K, N, R, L, spread, grads):
    p = _problem(M, K, N, R, L, seed=2 * M + R, spread=spread)
    plan = B.sq_lora_plan(p["ids"], L)
    _, _, t, _ = ref.lora_forward(p["x"], p["A"], p["B"], p["scale"], p["ids"], p["base"], BF)
    t = t.float()
    has = (p["ids"] >= 0) & (p["ids"] < L)
    t[~has] = float("nan")                  # never read
    dA, dB, dx = B.sq_lora_backward(p["dy"], p["x"], t, p["A"], p["B"], p["scale"], plan,
                                    p["dx_base"], grad_dtype=grads)
    want = ref.lora_backward(p["dy"], p["x"], t, p["A"], p["B"], p["scale"], p["ids"],
                             p["dx_base"], grads)
    assert dA.dtype == dB.dtype == grads
    for name, got in (("dA", dA), ("dB", dB), ("dx", dx)):
        ref.check(got, *want[name], name)
    for a in range(L):                      # an adapter without rows: exact zeros
        if not (p["ids"] == a).any():
            assert (dA[a] == 0).all() and (dB[a] == 0).all()
    assert torch.equal(dx[~has], p["dx_base"][~has])
    assert B.sq_get_device_status() == B.SQ_OK


def test_plan_orders_rows_by_adapter_and_keeps_their_order():
    for M, L, seed in ((0, 3, 1), (1, 1, 2), (1000, 7, 3), (70000, 1024, 4), (33, 1024, 5)):
        ids = torch.randint(-3, L + 3, (M,), generator=_gen(seed), device="cuda").to(torch.int32)
        plan = B.sq_lora_plan(ids, L).cpu().tolist()
        key = torch.where((ids >= 0) & (ids < L), ids, L).cpu()
        order = torch.sort(key, stable=True).indices.tolist()
        start = [0]
        for b in range(L + 1):
            start.append(start[-1] + int((key == b).sum()))
        assert plan[1:3] == [M, L]
        tiles = [(b, s) for b in range(L + 1) for s in range(start[b], start[b + 1], 128)]
        assert plan[3] == len(tiles)
        assert plan[4:4 + L + 2] == [sum(t[0] < b for t in tiles) for b in range(L + 2)]
        at = (4 + L + 2 + 3) // 4 * 4
        for b, s in tiles:     # {bin, rows, place, neighbours, row numbers}
            n = min(128, start[b + 1] - s)
            assert plan[at:at + 4] == [b, n, s, int(order[s + n - 1] - order[s] == n - 1)]
            assert plan[at + 4:at + 132] == order[s:s + n] + [order[s]] * (128 - n)
            at += 132


def test_in_place_strides_and_columns_beyond_are_untouched():
    """x, base and y as column slices of wider buffers; in place; a NaN in a row
    without an adapter and in the columns beyond stays where it is."""
    M, K, N, R, L = 150, 128, 264, 16, 3
    p = _problem(M, K, N, R, L, seed=9)
    wide = torch.full((M, K + 24), float("nan"), dtype=BF, device="cuda")
    wide[:, 8:8 + K] = p["x"]
    out = torch.full((M, 3 * N), 3.0, dtype=BF, device="cuda")
    out[:, N:2 * N] = p["base"]
    none = (p["ids"] < 0).nonzero()[:, 0]
    assert len(none) > 0
    wide[none] = float("nan")
    plan = B.sq_lora_plan(p["ids"], L)
    view = out[:, N:2 * N]
    y, t = B.sq_lora_forward(wide[:, 8:8 + K], p["A"], p["B"], p["scale"], plan, view, y=view)
    yr, ye, _, _ = ref.lora_forward(p["x"], p["A"], p["B"], p["scale"], p["ids"], p["base"], BF)
    ref.check(out[:, N:2 * N].contiguous(), yr, ye, "y")
    assert (out[:, :N] == 3.0).all() and (out[:, 2 * N:] == 3.0).all()
    dy = torch.full((M, N + 8), float("nan"), dtype=BF, device="cuda")
    dy[:, :N] = p["dy"]
    dy[none] = float("nan")
    dxw = torch.full((M, K + 16), 5.0, dtype=BF, device="cuda")
    dxw[:, :K] = p["dx_base"]
    tt = torch.nan_to_num(t)
    want = ref.lora_backward(p["dy"], p["x"], tt, p["A"], p["B"], p["scale"], p["ids"],
                             p["dx_base"], BF)
    dA, dB, dx = B.sq_lora_backward(dy[:, :N], wide[:, 8:8 + K], t, p["A"], p["B"], p["scale"],
                                    plan, dxw[:, :K], dx=dxw[:, :K])
    ref.check(dA, *want["dA"], "dA")
    ref.check(dB, *want["dB"], "dB")
    ref.check(dxw[:, :K].contiguous(), *want["dx"], "dx")
    assert (dxw[:, K:] == 5.0).all()


def test_parts_on_their_own():
    """No base: zeros; gradients of the weights only, or of the input only."""
    M, K, N, R, L = 90, 64, 80, 8, 2
    p = _problem(M, K, N, R, L, seed=3, spread="scattered")
    plan = B.sq_lora_plan(p["ids"], L)
    y, t = B.sq_lora_forward(p["x"], p["A"], p["B"], p["scale"], plan, None)
    yr, ye, _, _ = ref.lora_forward(p["x"], p["A"], p["B"], p["scale"], p["ids"], None, BF)
    ref.check(y, yr, ye, "y")
    a = (p["dy"], p["x"], t, p["A"], p["B"], p["scale"], plan)
    dA, dB, dx = B.sq_lora_backward(*a, None)
    dA1, dB1, none = B.sq_lora_backward(*a, None, need_dx=False)
    none2, none3, dx1 = B.sq_lora_backward(*a, None, need_weights=False)
    assert none is none2 is none3 is None
    assert torch.equal(dA, dA1) and torch.equal(dB, dB1) and torch.equal(dx, dx1)


def test_no_rows():
    A = torch.zeros(2, 8, 64, dtype=BF, device="cuda")
    Bm = torch.zeros(2, 72, 8, dtype=BF, device="cuda")
    s = torch.ones(2, device="cuda")
    x, dy = torch.empty(0, 64, dtype=BF, device="cuda"), torch.empty(0, 72, dtype=BF, device="cuda")
    plan = B.sq_lora_plan(torch.empty(0, dtype=torch.int32, device="cuda"), 2)
    y, t = B.sq_lora_forward(x, A, Bm, s, plan, None)
    assert y.shape == (0, 72)
    dA = torch.ones(2, 8, 64, dtype=BF, device="cuda")
    dA, dB, dx = B.sq_lora_backward(dy, x, t, A, Bm, s, plan, None, dA=dA)
    assert (dA == 0).all() and (dB == 0).all() and dx.shape == (0, 64)


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("R,spread", [(32, "runs"), (64, "mixed"), (128, "mixed"), (8, "one")])
def test_same_bits_every_time_and_from_a_graph(R, spread, out):
    """Fixed orders of all sums: repeated calls, another stream and a replayed
    graph give the same bits; new inputs in the captured buffers give theirs."""
    M, K, N, L = 2300, 640, 2296, 2
    p = _problem(M, K, N, R, L, seed=21, spread=spread, out=out)
    plan = B.sq_lora_plan(p["ids"], L)

    def call():
        y, t = B.sq_lora_forward(p["x"], p["A"], p["B"], p["scale"], plan, p["base"])
        return (y, *B.sq_lora_backward(p["dy"], p["x"], t, p["A"], p["B"], p["scale"], plan,
                                       p["dx_base"], grad_dtype=out))

    first = call()
    for _ in range(20):         # back to back, one call's kernels behind the other's
        again = call()
    for u, v in zip(first, again):
        assert torch.equal(u, v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = call()
    graph.replay()
    torch.cuda.synchronize()
    for u, v, w in zip(first, second, third):
        assert torch.equal(u, v) and torch.equal(u, w)
    p["x"].copy_(p["x"].flip(0))
    graph.replay()
    fresh = call()
    torch.cuda.synchronize()
    for u, w in zip(fresh, third):
        assert torch.equal(u, w)
    assert B.sq_get_device_status() == B.SQ_OK


def test_plan_of_another_batch_is_reported_and_nothing_written():
    M, K, N, R, L = 40, 64, 64, 8, 2
    p = _problem(M, K, N, R, L, seed=4)
    other = B.sq_lora_plan(torch.zeros(M + 1, dtype=torch.int32, device="cuda"), L)
    y = torch.full((M, N), 9.0, dtype=BF, device="cuda")
    # the binding refuses a plan of another size ...
    with pytest.raises(ValueError, match="plan"):
        B.sq_lora_forward(p["x"], p["A"], p["B"], p["scale"], B.sq_lora_plan(
            torch.zeros(400, dtype=torch.int32, device="cuda"), L), p["base"], y=y)
    # ... and the kernels one that says that it is not theirs
    t = torch.full((M, R), 9.0, device="cuda")
    B.sq_lora_forward(p["x"], p["A"], p["B"], p["scale"], other, p["base"], y=y, t=t)
    assert B.sq_get_device_status() == B.SQ_ERR_INVALID_ARG
    dA, dB, dx = (torch.full(s, 9.0, dtype=BF, device="cuda") for s in ((L, R, K), (L, N, R), (M, K)))
    B.sq_lora_backward(p["dy"], p["x"], t, p["A"], p["B"], p["scale"], other, p["dx_base"], dx=dx,
                       dA=dA, dB=dB)
    assert B.sq_get_device_status() == B.SQ_ERR_INVALID_ARG
    assert all((g == 9.0).all() for g in (dA, dB, dx))
    assert (y == 9.0).all() and (t == 9.0).all()
    assert B.sq_get_device_status() == B.SQ_OK


FEW = [  # M, K, N, R, L, spread: around the sizes up to which one kernel does both products
    (1, 8, 8, 8, 1, "one"), (2, 64, 4096, 64, 2, "one"), (15, 520, 264, 128, 1, "one"),
    (16, 1536, 1536, 16, 1, "one"), (17, 1536, 1536, 16, 1, "one"), (17, 264, 1000, 40, 2, "one"),
    (32, 2056, 72, 104, 9, "scattered"), (32, 1536, 2048, 128, 2, "one"), (33, 256, 64, 8, 3, "scattered"),
    (31, 72, 2056, 128, 40, "scattered"), (24, 128, 128, 16, 3, "none"), (9, 6144, 1536, 24, 1024, "runs"),
]


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,K,N,R,L,spread", FEW)
def test_few_rows(M, K, N, R, L, spread, out):
    """Strided and in place, zeros for base, rows without an adapter left alone,
    and the same bits again."""
    p = _problem(M, K, N, R, L, seed=3 * M + R, spread=spread, out=out)
    plan = B.sq_lora_plan(p["ids"], L)
    some = (p["ids"] >= 0) & (p["ids"] < L)
    wide = torch.full((M, N + 16), 3.25, dtype=out, device="cuda")
    y = wide[:, 8:8 + N]
    y.copy_(p["base"])
    x = torch.full((M, K + 8), float("nan"), dtype=BF, device="cuda")
    x[:, :K] = p["x"]
    t = torch.full((M, R), -7.5, device="cuda")
    B.sq_lora_forward(x[:, :K], p["A"], p["B"], p["scale"], plan, y, y=y, t=t)
    v, e, T, eT = ref.lora_forward(p["x"], p["A"], p["B"], p["scale"], p["ids"], p["base"], out)
    ref.check(y.contiguous(), v, e, "y")
    ref.check(t[some], T[some], eT[some], "t")
    assert (t[~some] == -7.5).all() and torch.equal(y[~some], p["base"][~some])
    assert (wide[:, :8] == 3.25).all() and (wide[:, 8 + N:] == 3.25).all()
    z, _ = B.sq_lora_forward(p["x"], p["A"], p["B"], p["scale"], plan, None,
                             y=torch.full((M, N), 9.0, dtype=out, device="cuda"))
    v, e, _, _ = ref.lora_forward(p["x"], p["A"], p["B"], p["scale"], p["ids"], None, out)
    ref.check(z, v, e, "y without base")
    again, _ = B.sq_lora_forward(p["x"], p["A"], p["B"], p["scale"], plan, p["base"])
    assert torch.equal(again, y)
    assert B.sq_get_device_status() == B.SQ_OK


def test_infinite_values_of_a_used_row_stay_infinite():
    """Places past a tile's last row add nothing, not even 0 times infinity."""
    M, K, N, R, L = 300, 128, 128, 16, 3
    p = _problem(M, K, N, R, L, seed=4, spread="scattered")
    first = int((p["ids"] == 1).nonzero()[0, 0])
    p["x"][first, 5] = float("inf")
    p["dy"][first, 7] = float("inf")
    plan = B.sq_lora_plan(p["ids"], L)
    t = torch.rand(M, R, device="cuda") + 0.5
    dA, dB, _ = B.sq_lora_backward(p["dy"], p["x"], t, p["A"], p["B"], p["scale"], plan, None,
                                   need_dx=False)
    # dy's infinity makes dt of that row infinite (NaN where B is 0): dA[1] whole
    assert torch.isinf(dB[1, 7]).all() and torch.isfinite(dB[1, :7]).all()
    assert torch.isfinite(dB[1, 8:]).all()
    assert torch.isfinite(dA[[0, 2]]).all() and torch.isfinite(dB[[0, 2]]).all()
    p["dy"][first, 7] = 1.0
    dA, dB, _ = B.sq_lora_backward(p["dy"], p["x"], t, p["A"], p["B"], p["scale"], plan, None,
                                   need_dx=False)
    assert torch.isinf(dA[1, :, 5]).all() and torch.isfinite(dB).all()
    assert torch.isfinite(dA[1, :, :5]).all() and torch.isfinite(dA[1, :, 6:]).all()


def test_the_stride_of_a_single_row_says_nothing():
    K, N, R, L = 64, 4096, 128, 2
    p = _problem(1, K, N, R, L, seed=8, spread="one")
    plan = B.sq_lora_plan(p["ids"], L)
    far = {k: torch.as_strided(p[k], p[k].shape, (2 ** 42, 1)) for k in ("x", "base", "dy")}
    y, t = B.sq_lora_forward(p["x"], p["A"], p["B"], p["scale"], plan, p["base"])
    z, _ = B.sq_lora_forward(far["x"], p["A"], p["B"], p["scale"], plan, far["base"])
    assert torch.equal(y, z)
    want = B.sq_lora_backward(p["dy"], p["x"], t, p["A"], p["B"], p["scale"], plan, p["dx_base"])
    got = B.sq_lora_backward(far["dy"], far["x"], t, p["A"], p["B"], p["scale"], plan,
                             torch.as_strided(p["dx_base"], (1, K), (2 ** 42, 1)))
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    wq, s_w = torch.ones(N, K, dtype=torch.int8, device="cuda"), torch.ones(1, N, device="cuda")
    assert torch.equal(B.sq_dualscale_seglinear_input_grad(p["dy"], wq, s_w, None, B.Segments()),
                       B.sq_dualscale_seglinear_input_grad(far["dy"], wq, s_w, None, B.Segments()))


def test_plans_made_by_two_threads_at_once():
    """Plans of one and of 1024 adapters, whose kernels need different amounts of
    shared memory, from two host threads."""
    import threading
    ids = torch.arange(500, device="cuda", dtype=torch.int32) % 7
    want = {L: B.sq_lora_plan(ids, L) for L in (1, 1024)}
    wrong = []

    def run(L):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(200):
                try:
                    got = B.sq_lora_plan(ids, L)
                except B.SegQuantError as e:
                    wrong.append((L, str(e)))
                    return
            torch.cuda.current_stream().synchronize()
            tiles = int(got[3])
            n = (4 + L + 2 + 3) // 4 * 4 + 132 * tiles
            head = 4 + L + 2
            if not (torch.equal(got[:head], want[L][:head])
                    and torch.equal(got[(4 + L + 2 + 3) // 4 * 4:n], want[L][(4 + L + 2 + 3) // 4 * 4:n])):
                wrong.append((L, "differs"))

    threads = [threading.Thread(target=run, args=(L,)) for L in (1, 1024)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong, wrong


@pytest.mark.parametrize("M,K,N,R,L,spread", [(333, 1536, 1536, 8, 3, "runs"),
                                              (6000, 1536, 2048, 64, 2, "mixed")])
def test_backward_kernels_side_by_side_keep_the_streams_order(M, K, N, R, L, spread):
    """dA, dB and dx are whole for whatever comes next on the stream: consumers
    right behind the call, and the buffers used again by the next one, eager and
    replayed, give the bits of calls that are waited for."""
    p = _problem(M, K, N, R, L, seed=21, spread=spread)
    plan = B.sq_lora_plan(p["ids"], L)
    _, t = B.sq_lora_forward(p["x"], p["A"], p["B"], p["scale"], plan, p["base"])
    ws = torch.empty(B.sq_lora_workspace_bytes(M, R, L), dtype=torch.uint8, device="cuda")
    dA, dB = torch.empty_like(p["A"]), torch.empty_like(p["B"])
    dx = torch.empty_like(p["x"])
    dys = [p["dy"], (2 * p["dy"].float()).to(BF), (-p["dy"].float()).to(BF)]

    def step(dy):
        B.sq_lora_backward(dy, p["x"], t, p["A"], p["B"], p["scale"], plan, None, dx=dx, dA=dA,
                           dB=dB, workspace=ws)
        return [v.clone() for v in (dA, dB, dx)]

    want = []
    for dy in dys:
        want.append(step(dy))
        torch.cuda.synchronize()
    for _ in range(20):
        got = [step(dy) for dy in dys]
        for a, b in zip(want, got):
            assert all(torch.equal(u, v) for u, v in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [step(dy) for dy in dys]
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("K,N,R", [(200, 328, 24), (1536, 520, 128)])
def test_requests_of_lengths_around_the_boxes(K, N, R, out):
    """Tiles put together from several requests: 32 and 64 neighbouring rows come
    as boxes wherever they begin, others row by row."""
    lengths = [31, 32, 33, 64, 1, 95, 63, 96, 65, 128, 7, 160, 32, 64, 130, 5, 224, 33]
    L = 3
    ids = torch.cat([torch.full((n,), i * 5 % (L + 1) - 1) for i, n in enumerate(lengths)])
    M = len(ids)
    p = _problem(M, K, N, R, L, seed=31, spread="one", out=out)
    p["ids"] = ids.to(torch.int32).cuda()
    plan = B.sq_lora_plan(p["ids"], L)
    y, t = B.sq_lora_forward(p["x"], p["A"], p["B"], p["scale"], plan, p["base"])
    v, e, T, eT = ref.lora_forward(p["x"], p["A"], p["B"], p["scale"], p["ids"], p["base"], out)
    some = p["ids"] >= 0
    ref.check(y, v, e, "y")
    ref.check(t[some], T[some], eT[some], "t")
    want = ref.lora_backward(p["dy"], p["x"], t, p["A"], p["B"], p["scale"], p["ids"], p["dx_base"],
                             out)
    got = B.sq_lora_backward(p["dy"], p["x"], t, p["A"], p["B"], p["scale"], plan, p["dx_base"],
                             grad_dtype=out)
    for name, value in zip(("dA", "dB", "dx"), got):
        ref.check(value, *want[name], name)
    assert B.sq_get_device_status() == B.SQ_OK
