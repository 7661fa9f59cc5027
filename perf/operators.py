"""The operators that stand around the quantized linear, each as a plain torch
computation and as the library's calls: low-rank adapters of many requests beside
a shared projection (forward, backward), rotary positions on the q|k columns of a
QKV projection (forward, backward), group norm with an activation on channels-last
features (forward, backward), and the input gradient of the frozen quantized linear.

`run` takes the plain form where `own` is false and the library's entry points
where it is true; `exact` restates each operator in 64 bits.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# --------------------------------------------------------------------- cases
def listed():
    return [
        # One token of each of 16 requests that use eight adapters in turn: the
        # latency of a served step beside a 1536-wide projection.
        dict(name="lora_fwd_decode", op="lora_forward", M=16, K=1536, N=1536, R=16, L=8,
             requests=16, out="bf16"),
        # A packed batch of ragged prompts, some perhaps without an adapter,
        # beside a projection with fp32 output rows.
        dict(name="lora_fwd_ragged", op="lora_forward", M=1501, K=1536, N=2304, R=48, L=5,
             requests=9, out="f32"),
        # The SD3.5 FFN's first linear with one adapter over the whole batch.
        dict(name="lora_fwd_ffn", op="lora_forward", M=8858, K=1536, N=6144, R=64, L=1,
             requests=1, out="bf16"),
        # Fine-tuning several small adapters at once on one text prompt's rows.
        dict(name="lora_bwd_small", op="lora_backward", M=333, K=1536, N=1536, R=8, L=3,
             requests=3, out="bf16"),
        # Fine-tuning two adapters beside the SD3.5 FFN's first linear.
        dict(name="lora_bwd_ffn", op="lora_backward", M=8858, K=1536, N=6144, R=64, L=2,
             requests=2, out="bf16"),
        # One decoding step far into a long context: half layout, part of the head.
        dict(name="rope_fwd_decode", op="rope_forward", M=24, H=32, D=64, rot=32,
             layout="half", axes=1, max_pos=1000000, out="bf16"),
        # FLUX-shaped q|k rows (24 + 24 heads of 128), interleaved, three axes, backward.
        dict(name="rope_bwd_image", op="rope_backward", M=9216, H=48, D=128, rot=128,
             layout="interleaved", axes=3, max_pos=4096, out="bf16"),
        # A U-Net's first level: 128 x 128 latents of 320 channels, SiLU.
        dict(name="gn_fwd_unet", op="group_norm_forward", B=2, S=16384, C=320, G=32, act="silu"),
        # An odd small latent at a deep level, without an activation (before a projection).
        dict(name="gn_fwd_small", op="group_norm_forward", B=1, S=391, C=1280, G=32, act="none"),
        # The backward pass at a U-Net's second level.
        dict(name="gn_bwd_unet", op="group_norm_backward", B=4, S=4096, C=640, G=32, act="silu"),
        # Input gradient of the attention out-projection: 24 input segments, divisors.
        dict(name="dgrad_outproj", op="input_grad", M=1109, N=1536, K=1536, segments=24,
             mode="input", divisor=True),
        # Input gradient of the SD3.5 FFN's first linear.
        dict(name="dgrad_ffn", op="input_grad", M=8858, N=6144, K=1536, segments=1,
             mode="none", divisor=False),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["lora_forward", "lora_forward", "lora_backward", "lora_backward",
                     "rope_forward", "rope_backward", "group_norm_forward",
                     "group_norm_backward", "input_grad"])
    if op.startswith("lora"):
        M = _log(rng, 1, 8000)
        R = rng.choice([8, 16, 24, 32, 48, 64])
        K, N = _log(rng, 64, 4096, 8), _log(rng, 64, 4096, 8)
        L = _log(rng, 1, 24) if M <= 1024 else rng.randint(1, 3)
        return dict(op=op, M=M, K=K, N=N, R=R, L=L, requests=min(M, _log(rng, 1, 64)),
                    out=rng.choice(["bf16", "bf16", "f32"]))
    if op.startswith("rope"):
        D = rng.choice([32, 64, 80, 96, 128])
        layout = rng.choice(["half", "interleaved"])
        axes = rng.choice([1, 1, 2, 3])
        rot = D if rng.random() < 0.5 else 16 * rng.randint(1, D // 16)
        return dict(op=op, M=_log(rng, 1, 9000), H=rng.randint(1, 40), D=D, rot=rot,
                    layout=layout, axes=axes, max_pos=_log(rng, 64, 1000000),
                    out=rng.choice(["bf16", "bf16", "f32"]))
    if op.startswith("group_norm"):
        G = rng.choice([1, 4, 8, 16, 32])
        C = G * 8 * rng.randint(1, 5) if G < 32 else 32 * rng.choice([4, 6, 10, 20, 24, 30, 40])
        return dict(op=op, B=rng.randint(1, 4), S=_log(rng, 1, 8192), C=C, G=G,
                    act=rng.choice(["none", "silu", "gelu"]))
    seg = rng.choice([1, 3, 6])
    mode = "none" if seg == 1 else rng.choice(["input", "output"])
    return dict(op=op, M=_log(rng, 1, 8000), N=384 * rng.randint(1, 10),
                K=192 * rng.randint(1, 10), segments=seg, mode=mode,
                divisor=rng.random() < 0.5)


# ------------------------------------------------------------------- prepare
def _pairs(case):
    """Rotated pairs of each axis: the axes share them, the first takes what is left."""
    n, a = case["rot"] // 2, case["axes"]
    rest = n // a
    return [n - rest * (a - 1)] + [rest] * (a - 1)


def prepare(case, seed):
    op = case["op"]
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def randint(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = dict(case=dict(case), op=op)
    if op.startswith("lora"):
        M, K, N, R, L = (case[k] for k in "MKNRL")
        s["x"] = (randn(M, K) * torch.exp(rand(K) * 1.8 - 0.7)).to(BF16)
        s["A"] = (randn(L, R, K) / math.sqrt(K)).to(BF16)
        s["B"] = (randn(L, N, R) * 0.1).to(BF16)
        s["scale"] = 0.5 + 1.5 * rand(L)
        # a packed batch: requests of ragged lengths (some empty), each with an
        # adapter or, one in eight where there are several, with none
        nr = case["requests"]
        if nr == M:
            request = torch.arange(M, device="cuda")
        else:
            cuts = torch.sort(randint(0, M + 1, nr - 1)).values
            request = torch.searchsorted(cuts, torch.arange(M, device="cuda"), right=True)
        of = (torch.arange(nr, device="cuda") + randint(0, L, 1)) % L
        if nr > 2:
            of = torch.where(rand(nr) < 0.125, -1, of)
        s["ids"] = of[request].to(torch.int32)
        if own:
            # The batch's row order by adapter: made once per batch, shared by
            # every adapted layer that the batch goes through.
            from w8a8_gemm_b200 import binding as sq
            s["plan"] = sq.sq_lora_plan(s["ids"], L)
        if op == "lora_forward":
            s["base"] = randn(M, N).to(BF16 if case["out"] == "bf16" else F32)
        else:
            s["dy"] = randn(M, N).to(BF16)
            s["base"] = randn(M, K).to(BF16)
            s["t"] = (s["x"].float() @ s["A"].float().reshape(L * R, K).t()
                      * _onehot(s["ids"], L, R)).reshape(M, L, R).sum(1)
    elif op.startswith("rope"):
        M, H, D, rot = case["M"], case["H"], case["D"], case["rot"]
        s["x"] = randn(M, H * D).to(BF16 if case["out"] == "bf16" else F32)
        s["positions"] = randint(0, case["max_pos"], M, case["axes"]).to(torch.int32)
        freq = []
        for n in _pairs(case):
            freq += [10000.0 ** (-i / max(n, 1)) for i in range(n)]
        s["inv_freq"] = torch.tensor(freq, dtype=F64, device="cuda").to(F32)
        s["axis"] = torch.tensor([a for a, n in enumerate(_pairs(case)) for _ in range(n)],
                                 device="cuda")
        s["factor"] = 1.0 if case["max_pos"] < 100000 else 1.25
    elif op.startswith("group_norm"):
        B, S, C = case["B"], case["S"], case["C"]
        s["x"] = (randn(B, S, C) * (0.3 + 2 * rand(C)) + 2 * randn(C)).to(BF16)
        s["gamma"] = (1 + 0.2 * randn(C)).to(BF16)
        s["beta"] = (0.2 * randn(C)).to(BF16)
        s["eps"] = 1e-5
        if op == "group_norm_backward":
            s["dy"] = randn(B, S, C).to(BF16)
            # the statistics that the forward pass kept
            xg = s["x"].double().reshape(B, S, case["G"], -1)
            mean = xg.mean((1, 3))
            var = (xg - mean[:, None, :, None]).square().mean((1, 3))
            s["mean"], s["rstd"] = mean.float(), torch.rsqrt(var + s["eps"]).float()
    else:
        M, N, K, n = case["M"], case["N"], case["K"], case["segments"]
        s["dy"] = randn(M, N).to(BF16)
        s["wq"] = randint(-127, 128, N, K).to(torch.int8)
        S = n if case["mode"] == "input" else 1
        s["s_w"] = 0.0002 * torch.exp(rand(S, N) * 2)
        extent = {"none": 1, "input": K, "output": N}[case["mode"]]
        s["offsets"] = None if case["mode"] == "none" else [extent * i // n for i in range(n + 1)]
        s["d"] = torch.exp(2 * rand(1, K) - 1) if case["divisor"] else None
    return s


# ------------------------------------------------------------- plain operators
def _onehot(ids, L, R):
    """[M][L*R]: one where the row's adapter is the column's."""
    hit = ids[:, None] == torch.arange(L, device=ids.device)[None]
    return hit.float().repeat_interleave(R, 1)


def _lora_forward(s):
    L, R, K = s["A"].shape
    N = s["B"].shape[1]
    a = s["A"].float().reshape(L * R, K)
    b = s["B"].float().permute(0, 2, 1).reshape(L * R, N)
    t = (s["x"].float() @ a.t()) * _onehot(s["ids"], L, R) * s["scale"].repeat_interleave(R)
    return {"y": (s["base"].float() + t @ b).to(s["base"].dtype)}


def _lora_backward(s):
    L, R, K = s["A"].shape
    N = s["B"].shape[1]
    dy, x = s["dy"].float(), s["x"].float()
    a = s["A"].float().reshape(L * R, K)
    b = s["B"].float().permute(0, 2, 1).reshape(L * R, N)
    w = _onehot(s["ids"], L, R) * s["scale"].repeat_interleave(R)
    dt = (dy @ b.t()) * w
    t = s["t"].repeat(1, L) * w
    kind = BF16 if s["case"]["out"] == "bf16" else F32
    return {"dA": (dt.t() @ x).reshape(L, R, K).to(kind),
            "dB": (t.t() @ dy).reshape(L, R, N).permute(0, 2, 1).contiguous().to(kind),
            "dx": (s["base"].float() + dt @ a).to(BF16)}


def _rope(s, sign):
    c = s["case"]
    M, H, D, rot = c["M"], c["H"], c["D"], c["rot"]
    # far positions: the angle needs more than 24 bits before it is reduced
    angle = s["positions"].double()[:, s["axis"]] * s["inv_freq"].double()
    cos = (s["factor"] * angle.cos()).float()[:, None]
    sin = (sign * s["factor"] * angle.sin()).float()[:, None]
    x = s["x"].float().reshape(M, H, D)
    if c["layout"] == "half":
        u, v = x[..., :rot // 2], x[..., rot // 2:rot]
        r = torch.cat([u * cos - v * sin, u * sin + v * cos], -1)
    else:
        u, v = x[..., 0:rot:2], x[..., 1:rot:2]
        r = torch.stack([u * cos - v * sin, u * sin + v * cos], -1).reshape(M, H, rot)
    return {"y": torch.cat([r, x[..., rot:]], -1).reshape(M, H * D).to(s["x"].dtype)}


def _act(v, act):
    """act(v) and its derivative."""
    if act == "none":
        return v, torch.ones_like(v)
    if act == "silu":
        g = torch.sigmoid(v)
        return v * g, g * (1 + v * (1 - g))
    k = math.sqrt(2 / math.pi)
    th = torch.tanh(k * (v + 0.044715 * v * v * v))
    d = 0.5 * (1 + th) + 0.5 * v * (1 - th * th) * k * (1 + 3 * 0.044715 * v * v)
    return 0.5 * v * (1 + th), d


def _group_norm_forward(s):
    c = s["case"]
    B, S, C = s["x"].shape
    x = s["x"].float().reshape(B, S, c["G"], -1)
    mean = x.mean((1, 3), keepdim=True)
    var = (x - mean).square().mean((1, 3), keepdim=True)
    rstd = torch.rsqrt(var + s["eps"])
    v = ((x - mean) * rstd).reshape(B, S, C) * s["gamma"].float() + s["beta"].float()
    return {"y": _act(v, c["act"])[0].to(BF16), "mean": mean.reshape(B, -1),
            "rstd": rstd.reshape(B, -1)}


def _group_norm_backward(s):
    c = s["case"]
    B, S, C = s["x"].shape
    G = c["G"]
    n = S * C // G
    xh = ((s["x"].float().reshape(B, S, G, -1) - s["mean"][:, None, :, None])
          * s["rstd"][:, None, :, None])
    gamma = s["gamma"].float()
    v = xh.reshape(B, S, C) * gamma + s["beta"].float()
    dv = s["dy"].float() * _act(v, c["act"])[1]
    h = (dv * gamma).reshape(B, S, G, -1)
    s1 = (h * xh).sum((1, 3), keepdim=True)
    s2 = h.sum((1, 3), keepdim=True)
    dx = s["rstd"][:, None, :, None] * (h - (s2 + xh * s1) / n)
    return {"dx": dx.reshape(B, S, C).to(BF16),
            "dgamma": (dv * xh.reshape(B, S, C)).sum((0, 1)).to(BF16),
            "dbeta": dv.sum((0, 1)).to(BF16)}


def _input_grad(s):
    c = s["case"]
    w = s["wq"].float()
    if c["mode"] == "input":
        seg = torch.bucketize(torch.arange(c["K"], device=w.device),
                              torch.tensor(s["offsets"][1:], device=w.device), right=True)
        w = w * s["s_w"][seg].t()
    else:
        w = w * s["s_w"][0][:, None]
    if s["d"] is not None:
        w = w / s["d"]
    return {"dx": (s["dy"].float() @ w).to(BF16)}


def _plain(s):
    op = s["op"]
    if op == "lora_forward":
        return _lora_forward(s)
    if op == "lora_backward":
        return _lora_backward(s)
    if op == "rope_forward":
        return _rope(s, 1.0)
    if op == "rope_backward":
        return _rope(s, -1.0)
    if op == "group_norm_forward":
        return _group_norm_forward(s)
    if op == "group_norm_backward":
        return _group_norm_backward(s)
    return _input_grad(s)


# ------------------------------------------------------------- library's calls
def _own(s):
    from w8a8_gemm_b200 import binding as sq
    c, op = s["case"], s["op"]
    if op == "lora_forward":
        y, _ = sq.sq_lora_forward(s["x"], s["A"], s["B"], s["scale"], s["plan"], s["base"])
        return {"y": y}
    if op == "lora_backward":
        dA, dB, dx = sq.sq_lora_backward(s["dy"], s["x"], s["t"], s["A"], s["B"], s["scale"],
                                         s["plan"], s["base"],
                                         grad_dtype=BF16 if c["out"] == "bf16" else F32)
        return {"dA": dA, "dB": dB, "dx": dx}
    if op.startswith("rope"):
        f = sq.sq_rope_forward if op == "rope_forward" else sq.sq_rope_backward
        layout = (sq.SQ_ROPE_HALF if c["layout"] == "half" else sq.SQ_ROPE_INTERLEAVED)
        return {"y": f(s["x"], s["positions"], s["inv_freq"], c["D"], layout=layout,
                       axis_pairs=_pairs(c), factor=s["factor"])}
    if op.startswith("group_norm"):
        act = {"none": sq.SQ_ACT_NONE, "silu": sq.SQ_ACT_SILU, "gelu": sq.SQ_ACT_GELU}[c["act"]]
        if op == "group_norm_forward":
            y, mean, rstd = sq.sq_group_norm_forward(s["x"], c["G"], s["gamma"], s["beta"],
                                                     eps=s["eps"], act=act)
            return {"y": y, "mean": mean, "rstd": rstd}
        dx, dgamma, dbeta = sq.sq_group_norm_backward(s["dy"], s["x"], c["G"], s["gamma"],
                                                      s["beta"], s["mean"], s["rstd"], act=act)
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    mode = {"none": sq.SQ_SEG_NONE, "input": sq.SQ_SEG_INPUT, "output": sq.SQ_SEG_OUTPUT}
    seg = sq.Segments(mode[c["mode"]], s["offsets"])
    return {"dx": sq.sq_dualscale_seglinear_input_grad(s["dy"], s["wq"], s["s_w"], s["d"], seg)}


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op.startswith("lora"):
        M, K, N, R, L = (case[k] for k in "MKNRL")
        used = min(L, case["requests"])
        weights = 2 * used * R * (K + N)
        if op == "lora_forward":
            e = 2 if case["out"] == "bf16" else 4
            return {"bytes": 2 * M * K + 2 * e * M * N + weights + 4 * M,
                    "flops": 2 * M * R * (K + N)}
        g = (2 if case["out"] == "bf16" else 4) * L * R * (K + N)
        return {"bytes": 2 * M * N + 6 * M * K + 4 * M * R + weights + g + 4 * M,
                "flops": 4 * M * R * (K + N)}
    if op.startswith("rope"):
        e = 2 if case["out"] == "bf16" else 4
        n = case["M"] * case["H"] * case["D"]
        return {"bytes": 2 * e * n + 4 * case["M"] * case["axes"],
                "flops": 3 * case["M"] * case["H"] * case["rot"]}
    if op.startswith("group_norm"):
        n = case["B"] * case["S"] * case["C"]
        if op == "group_norm_forward":
            return {"bytes": 4 * n + 4 * case["C"], "flops": 10 * n}
        return {"bytes": 6 * n + 8 * case["C"], "flops": 25 * n}
    M, N, K = case["M"], case["N"], case["K"]
    return {"bytes": 2 * M * (N + K) + N * K, "flops": 2 * M * N * K}


# ---------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("lora"):
        return _exact_lora(case, s)
    if op.startswith("rope"):
        return _exact_rope(case, s)
    if op.startswith("group_norm"):
        return _exact_group_norm(case, s)
    w = s["wq"].double()
    if case["mode"] == "input":
        for i in range(case["segments"]):
            lo, hi = s["offsets"][i], s["offsets"][i + 1]
            w[:, lo:hi] *= s["s_w"][i].double()[:, None]
    else:
        w *= s["s_w"].double().reshape(-1, 1)
    if s["d"] is not None:
        w /= s["d"].double()
    return {"dx": torch.einsum("mn,nk->mk", s["dy"].double(), w)}


def _exact_lora(case, s):
    """Adapter by adapter, on the rows that have it."""
    out = {}
    if case["op"] == "lora_forward":
        out["y"] = s["base"].double()
    else:
        out = {"dA": torch.zeros_like(s["A"], dtype=F64), "dB": torch.zeros_like(s["B"], dtype=F64),
               "dx": s["base"].double()}
    for a in range(case["L"]):
        rows = (s["ids"] == a).nonzero()[:, 0]
        A, B, c = s["A"][a].double(), s["B"][a].double(), s["scale"][a].double()
        x = s["x"][rows].double()
        if case["op"] == "lora_forward":
            out["y"][rows] += c * torch.mm(torch.mm(x, A.t()), B.t())
        else:
            dy = s["dy"][rows].double()
            dt = c * torch.mm(dy, B)
            out["dB"][a] = c * torch.mm(dy.t(), s["t"][rows].double())
            out["dA"][a] = torch.mm(dt.t(), x)
            out["dx"][rows] += torch.mm(dt, A)
    return out


def _exact_rope(case, s):
    """Complex rotation of each pair."""
    M, H, D, rot = case["M"], case["H"], case["D"], case["rot"]
    z = s["x"].double().reshape(M, H, D)
    turn = torch.zeros(M, rot // 2, dtype=F64, device=z.device)
    at = 0
    for a, n in enumerate(_pairs(case)):
        turn[:, at:at + n] = (s["positions"][:, a:a + 1].double()
                              * s["inv_freq"][at:at + n].double())
        at += n
    if case["op"] == "rope_backward":
        turn = -turn
    w = s["factor"] * torch.exp(1j * turn)[:, None]
    out = z.clone()
    first, second = ((slice(0, rot // 2), slice(rot // 2, rot)) if case["layout"] == "half"
                     else (slice(0, rot, 2), slice(1, rot, 2)))
    r = torch.complex(z[..., first].contiguous(), z[..., second].contiguous()) * w
    out[..., first], out[..., second] = r.real, r.imag
    return {"y": out.reshape(M, H * D)}


def _exact_group_norm(case, s):
    """Through torch's differentiation of the definition, in 64 bits."""
    B, S, C, G = case["B"], case["S"], case["C"], case["G"]
    back = case["op"] == "group_norm_backward"
    x = s["x"].double().requires_grad_(back)
    gamma = s["gamma"].double().requires_grad_(back)
    beta = s["beta"].double().requires_grad_(back)
    var, mean = torch.var_mean(x.reshape(B, S, G, C // G), (1, 3), unbiased=False)
    rstd = 1 / (var + s["eps"]).sqrt()

    def wide(t):
        return t.repeat_interleave(C // G, 1)[:, None]

    v = (x - wide(mean)) * wide(rstd) * gamma + beta
    if case["act"] == "silu":
        v = v / (1 + torch.exp(-v))
    elif case["act"] == "gelu":
        v = 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if not back:
        return {"y": v, "mean": mean, "rstd": rstd}
    dx, dgamma, dbeta = torch.autograd.grad(v, (x, gamma, beta), s["dy"].double())
    return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
