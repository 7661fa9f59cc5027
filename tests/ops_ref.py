"""64-bit references of the operators around the quantized linear, each with an
elementwise bound on what its kernel may be off by.

The bounds count roundings.  U[t] = finfo(t).eps / 2 is the largest relative
error of one rounding to type t (bf16 2^-8, fp32 2^-24).  ACC(n) bounds a sum of
n products in fp32, relative to the sum of their magnitudes: n steps of at most
2^-23 each, a whole step of the fp32 grid rather than half of one, since the
matrix units need not round to nearest."""
import math

import torch

F64 = torch.float64
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = 1e-37   # below the smallest normal number a flush to zero may happen


def ACC(n):
    return n * 2.0 ** -23


def check(got, ref, bound, name):
    """got (any float type) within `bound` plus its own rounding of ref."""
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    g = got.detach().to(F64)
    assert torch.isfinite(g).all(), f"{name}: not finite"
    allowed = bound + U[got.dtype] * (ref.abs() + bound) + TINY
    excess = (g - ref).abs() / allowed
    worst = float(excess.max()) if excess.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3g} times the bound at {int(excess.argmax())}"


# ------------------------------------------------------------------ adapters
def lora_forward(x, A, B, scale, ids, base, out_dtype):
    """(y, bound, t, t bound); rows without an adapter keep base, t 0."""
    M, L, R = x.shape[0], A.shape[0], A.shape[1]
    K, N = A.shape[2], B.shape[1]
    dev = x.device
    y = torch.zeros(M, N, dtype=F64, device=dev) if base is None else base.to(F64).clone()
    e = torch.zeros_like(y)
    T = torch.zeros(M, R, dtype=F64, device=dev)
    eT = torch.zeros_like(T)
    ut = U[torch.bfloat16] if out_dtype == torch.bfloat16 else 2.0 ** -23
    for a in range(L):
        r = (ids == a).nonzero()[:, 0]
        xa, Aa, Ba, c = x[r].to(F64), A[a].to(F64), B[a].to(F64), float(scale[a])
        t = xa @ Aa.t()
        et = ACC(K + 8) * (xa.abs() @ Aa.abs().t())
        T[r], eT[r] = t, et
        et2 = et + ut * (t.abs() + et)
        d = c * (t @ Ba.t())
        ed = abs(c) * (et2 @ Ba.abs().t() + ACC(3 * R) * (t.abs() @ Ba.abs().t()))
        e[r] = ed + 2.0 ** -23 * (y[r].abs() + d.abs())
        y[r] += d
    return y, e, T, eT


def lora_backward(dy, x, t, A, B, scale, ids, dx_base, grad_dtype):
    """{name: (value, bound)} of dA, dB, dx; t as given (fp32)."""
    M, L, R, K, N = x.shape[0], A.shape[0], A.shape[1], A.shape[2], B.shape[1]
    dev = x.device
    ug = U[torch.bfloat16] if grad_dtype == torch.bfloat16 else 2.0 ** -23
    ub = U[torch.bfloat16]
    dA = torch.zeros(L, R, K, dtype=F64, device=dev)
    dB = torch.zeros(L, N, R, dtype=F64, device=dev)
    eA, eB = torch.zeros_like(dA), torch.zeros_like(dB)
    dx = torch.zeros(M, K, dtype=F64, device=dev) if dx_base is None else dx_base.to(F64).clone()
    ex = torch.zeros_like(dx)
    for a in range(L):
        r = (ids == a).nonzero()[:, 0]
        n = len(r)
        g, xa, ta = dy[r].to(F64), x[r].to(F64), t[r].to(F64)
        Aa, Ba, c = A[a].to(F64), B[a].to(F64), float(scale[a])
        dt = c * (g @ Ba)
        edt = abs(c) * ACC(N + 8) * (g.abs() @ Ba.abs()) + 2.0 ** -23 * dt.abs()
        dB[a] = c * (g.t() @ ta)
        eB[a] = abs(c) * (ug + ACC(3 * n + 8)) * (g.abs().t() @ ta.abs())
        dA[a] = dt.t() @ xa
        eA[a] = (edt + (ug + ACC(3 * n + 8)) * (dt.abs() + edt)).t() @ xa.abs()
        d = dt @ Aa
        ed = (edt + (ub + ACC(R)) * (dt.abs() + edt)) @ Aa.abs()
        ex[r] = ed + 2.0 ** -23 * (dx[r].abs() + d.abs())
        dx[r] += d
    return {"dA": (dA, eA), "dB": (dB, eB), "dx": (dx, ex)}


# -------------------------------------------------------------------- rotary
def rope(x, positions, inv_freq, D, layout, axis_pairs, factor, sign):
    """(y, bound); layout 0 interleaved, 1 half."""
    M, cols = x.shape
    H, rot = cols // D, 2 * inv_freq.numel()
    pos = positions.reshape(M, -1).to(F64)
    axis = torch.zeros(rot // 2, dtype=torch.long, device=x.device)
    at = 0
    for a, n in enumerate(axis_pairs or [rot // 2]):
        axis[at:at + n] = a
        at += n
    phi = sign * pos[:, axis] * inv_freq.to(F64)
    c, s = (factor * phi.cos())[:, None], (factor * phi.sin())[:, None]
    z = x.to(F64).reshape(M, H, D)
    y, e = z.clone(), torch.zeros_like(z)
    i = torch.arange(rot // 2, device=x.device)
    iu, iv = (i, i + rot // 2) if layout == 1 else (2 * i, 2 * i + 1)
    u, v = z[..., iu], z[..., iv]
    y[..., iu], y[..., iv] = u * c - v * s, u * s + v * c
    # the fraction of a turn rounds to fp32 (2^-25 turns, 1.9e-7 rad), sine and
    # cosine are within 2 steps of 2^-24, the factor and two products round
    b = abs(factor) * (u.abs() + v.abs()) * 2.0 ** -20
    e[..., iu], e[..., iv] = b, b
    return y.reshape(M, cols), e.reshape(M, cols)


# ---------------------------------------------------------------- group norm
def act(v, kind):
    """(value, first derivative) of SQ_ACT_NONE, _SILU, _GELU."""
    if kind == 0:
        return v, torch.ones_like(v)
    if kind == 1:
        g = torch.sigmoid(v)
        return v * g, g * (1 + v * (1 - g))
    k = math.sqrt(2 / math.pi)
    th = torch.tanh(k * (v + 0.044715 * v ** 3))
    return 0.5 * v * (1 + th), 0.5 * (1 + th) + 0.5 * v * (1 - th * th) * k * (1 + 0.134145 * v * v)


# e^x in fp32 is off by about 2^-21 (1 + |x|), at arguments that matter (where the
# derivative is not yet flat) |x| < 20: 2^-16 covers it and the few operations after it
ACT_EVAL = 2.0 ** -16


def _per_channel(p, C):
    """[B][G] -> [B][1][C]"""
    return p.to(F64).repeat_interleave(C // p.shape[1], 1)[:, None]


def group_norm_forward(x, G, gamma, beta, eps, kind):
    """(y, bound), (mean, bound), (rstd, bound)."""
    B, S, C = x.shape
    z = x.to(F64)
    zg = z.reshape(B, S, G, C // G)
    mean = zg.mean((1, 3))
    var = (zg - mean[:, None, :, None]).square().mean((1, 3))
    rstd = 1 / (var + eps).sqrt()
    big = zg.abs().amax((1, 3))
    # at most 2^7 roundings of values up to `big` lie between a value and the mean
    em = 2.0 ** -17 * big
    delta = em * rstd
    er = rstd * (2.0 ** -16 + delta)
    gm = torch.ones(C, dtype=F64, device=x.device) if gamma is None else gamma.to(F64)
    bt = torch.zeros(C, dtype=F64, device=x.device) if beta is None else beta.to(F64)
    xh = (z - _per_channel(mean, C)) * _per_channel(rstd, C)
    dl = _per_channel(delta, C)
    exh = dl + xh.abs() * (2.0 ** -16 + dl)
    v = xh * gm + bt
    ev = gm.abs() * exh + 2.0 ** -22 * (v.abs() + bt.abs())
    y, _ = act(v, kind)
    return ((y, 1.13 * ev + (ACT_EVAL * (1 + v.abs()) if kind else 0.0)), (mean, em),
            (rstd, er))


def group_norm_backward(dy, x, G, gamma, beta, mean, rstd, kind):
    """{name: (value, bound)} of dx, dgamma, dbeta from the given fp32 statistics."""
    B, S, C = x.shape
    n = S * C // G
    mu, rs = _per_channel(mean, C), _per_channel(rstd, C)
    gm = torch.ones(C, dtype=F64, device=x.device) if gamma is None else gamma.to(F64)
    bt = torch.zeros(C, dtype=F64, device=x.device) if beta is None else beta.to(F64)
    xh = (x.to(F64) - mu) * rs
    exh = 2.0 ** -22 * xh.abs()
    v = xh * gm + bt
    g, d1 = dy.to(F64), act(v, kind)[1]
    dv = g * d1
    # the derivative's slope is below 1.2 everywhere
    edv = g.abs() * ((ACT_EVAL if kind else 0.0)
                     + 1.2 * (gm.abs() * exh + 2.0 ** -22 * (v.abs() + bt.abs())) * (kind != 0)
                     + 2.0 ** -22 * d1.abs())
    su = 2.0 ** -15   # sums: at most 2^8 steps in a row, products rounded

    def over_group(t):
        return t.reshape(B, S, G, C // G).sum((1, 3))

    h = dv * gm
    eh = edv * gm.abs() + 2.0 ** -22 * h.abs()
    m1, m2 = over_group(h) / n, over_group(h * xh) / n
    e1 = over_group(eh + su * h.abs()) / n
    e2 = over_group(eh * xh.abs() + h.abs() * exh + su * (h * xh).abs()) / n
    m1, m2, e1, e2 = (_per_channel(t, C) for t in (m1, m2, e1, e2))
    dx = rs * (h - m1 - xh * m2)
    ex = rs * (eh + e1 + xh.abs() * e2 + exh * m2.abs()
               + 2.0 ** -21 * (h.abs() + m1.abs() + (xh * m2).abs()))
    return {"dx": (dx, ex),
            "dgamma": ((dv * xh).sum((0, 1)),
                       (edv * xh.abs() + dv.abs() * exh + su * (dv * xh).abs()).sum((0, 1))),
            "dbeta": (dv.sum((0, 1)), (edv + su * dv.abs()).sum((0, 1)))}


# ----------------------------------------------------------- input gradient
def dequantized(wq_values, s_w, d, mode, offsets, G):
    """W~ [N][K] in 64 bits; wq_values: the codes' values [N][K]."""
    w = wq_values.to(F64).clone()
    if mode == 2:
        for i in range(len(offsets) - 1):
            w[:, offsets[i]:offsets[i + 1]] *= s_w[i].to(F64)[:, None]
    else:
        w *= s_w[0].to(F64)[:, None]
    if d is not None:
        if G == 1:
            w /= d[0].to(F64)
        else:
            for g in range(G):
                w[offsets[g]:offsets[g + 1]] /= d[g].to(F64)
    return w


def input_grad(dy, w):
    """(dx, bound): W~ is rounded to bf16 after two fp32 operations."""
    g = dy.to(F64)
    return g @ w, (U[torch.bfloat16] * 1.001 + 2.0 ** -22 + ACC(dy.shape[1] + 8)) * (
        g.abs() @ w.abs())
