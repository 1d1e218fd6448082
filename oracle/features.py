"""Plain fp64 evaluation of the feature operators (group norm with an activation, rotary positions, cross attention),
their gradients by the written formulas, and the error bounds their float kernels are held to.

Everything runs on CPU torch tensors in float64 and shares no code with the library. tests/test_oracle_features.py
checks the gradients against automatic differentiation and central differences of the forward definitions.
"""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24  # half an ulp of float32, relative
ROUND = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126}  # subnormal rounding


def act(z, kind):
    return z if kind == "none" else z.clamp_min(0) if kind == "relu" else z / (1 + torch.exp(-z))


def act_slope(z, kind):
    if kind == "none":
        return torch.ones_like(z)
    if kind == "relu":
        return (z > 0).double()
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def group_norm(x, gamma, beta, groups, eps, kind, dy=None):
    """x [N, P, C] float64 (gamma, beta [C] or None). Returns a dict of y, mean, rstd [N, G] and, with dy, dx, dgamma,
    dbeta, each with a bound on the float32 kernels' error before the result's own rounding."""
    N, P, C = x.shape
    k = C // groups
    gamma = torch.ones(C, dtype=torch.float64) if gamma is None else gamma
    beta = torch.zeros(C, dtype=torch.float64) if beta is None else beta
    xg = x.reshape(N, P, groups, k)
    mean = xg.mean((1, 3))
    var = (xg - mean[:, None, :, None]).square().mean((1, 3))
    rstd = 1 / torch.sqrt(var + eps)
    wide = lambda t: t.repeat_interleave(k, 1)[:, None, :]  # noqa: E731  [N, G] -> [N, 1, C]
    xh = (x - wide(mean)) * wide(rstd)
    z = xh * gamma + beta
    # Statistics: sums over trees of short float32 runs, about 64 roundings deep at the sizes tested, relative to the
    # mean of |x| (mean) and to the variance; the mean's error moves every xh of its group alike.
    e = 64 * U32
    top = xg.abs().mean((1, 3))
    e_mean = e * (top - mean.abs()).clamp_min(0) / 8 + 4 * U32 * top
    e_rstd = 0.5 * e + 4 * U32 + (e_mean * rstd).square()
    e_xh = wide(e_mean * rstd) + xh.abs() * wide(e_rstd) + 4 * U32 * (xh.abs() + wide(mean.abs() * rstd) / 2)
    e_z = e_xh * gamma.abs() + 4 * U32 * (xh * gamma).abs() + 2 * U32 * z.abs()
    # the sigmoid: exponential and reciprocal within a few ulp, the exponent's rounding |z| ulp
    e_act = 0 if kind == "none" else U32 * (8 + 2 * z.abs())
    out = {"y": act(z, kind), "mean": mean, "rstd": rstd, "e_mean": e_mean + U32 * mean.abs(), "e_rstd": e_rstd * rstd}
    out["e_y"] = 1.1 * e_z + e_act * act(z, kind).abs()
    if dy is not None:
        slope = act_slope(z, kind)
        dz = dy * slope
        e_dz = dy.abs() * (0.5 * e_z + e_act * (slope.abs() + (0.25 if kind == "silu" else 0))) + 2 * U32 * dz.abs()
        if kind == "relu":  # the sign of a z within its own error is not determined
            e_dz = e_dz + dy.abs() * (z.abs() <= e_z)
        dh = dz * gamma
        group_mean = lambda t: wide(t.reshape(N, P, groups, k).mean((1, 3)))  # noqa: E731
        out["dgamma"], out["dbeta"] = (dz * xh).sum((0, 1)), dz.sum((0, 1))
        out["e_dgamma"] = (e_dz * xh.abs() + dz.abs() * e_xh + e * (dz * xh).abs()).sum((0, 1))
        out["e_dbeta"] = (e_dz + e * dz.abs()).sum((0, 1))
        m1, m2 = group_mean(dh), group_mean(dh * xh)
        out["dx"] = wide(rstd) * (dh - m1 - xh * m2)
        e_m1 = group_mean(e_dz * gamma.abs() + e * dh.abs())
        e_m2 = group_mean(e_dz * (gamma * xh).abs() + dh.abs() * e_xh + e * (dh * xh).abs())
        size = dh.abs() + m1.abs() + (xh * m2).abs()
        out["e_dx"] = wide(rstd) * (e_dz * gamma.abs() + e_m1 + e_xh * m2.abs() + xh.abs() * e_m2 + 8 * U32 * size
                                    + wide(e_rstd) * size)
    return out


def rotary(x, positions, axis_pairs, base, halves, back=False):
    """x [B, T, H, D] float64, positions [B or 1, T, A] float64. Returns (out, bound before rounding)."""
    n = sum(axis_pairs)
    angle = torch.cat([positions[:, :, a, None] * torch.tensor([base ** (-i / p) for i in range(p)],
                                                               dtype=torch.float64)
                       for a, p in enumerate(axis_pairs)], -1)[:, :, None, :]
    c, s = torch.cos(angle), torch.sin(-angle if back else angle)
    out = x.clone()
    at, to = (slice(0, n), slice(n, 2 * n)) if halves else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    u, v = x[..., at], x[..., to]
    out[..., at], out[..., to] = u * c - v * s, u * s + v * c
    # the reduced angle is within 2^-24 of a turn (two roundings), its sine and cosine within 2 ulp of one more, the
    # products and their sum round three times
    e = torch.zeros_like(x)
    e[..., at] = e[..., to] = (2 * math.pi + 4 + 3) * U32 * (u.abs() + v.abs())
    return out, e


def attention(q, k, v, scale, dtype, lengths=None, mask=None, do=None):
    """q [B, Tq, H, D], k, v [B, Tk, Hk, D] float64; mask bool, broadcastable to [B, H, Tq, Tk]. Returns a dict of o, lse
    and, with do, dq, dk, dv, each with the bound "e_" on a kernel's result (the result's own rounding included): sums
    and statistics in float32, the probabilities and score gradients rounded once to `dtype`."""
    B, Tq, H, D = q.shape
    Tk, Hk = k.shape[1], k.shape[2]
    u = ROUND[dtype] if dtype != torch.float32 else 0.0
    seen = torch.ones((B, H, Tq, Tk), dtype=torch.bool)
    if lengths is not None:
        seen &= torch.arange(Tk) < torch.as_tensor(lengths).clamp(0, Tk)[:, None, None, None]
    if mask is not None:
        seen &= mask
    some = seen.any(-1)
    anyrow, anykey = some, seen.reshape(B, Hk, H // Hk * Tq, Tk).any(2)
    # what lies where nothing looks changes nothing
    kh = torch.where(anykey[..., None], k.transpose(1, 2), 0.0).repeat_interleave(H // Hk, 1)
    vh = torch.where(anykey[..., None], v.transpose(1, 2), 0.0).repeat_interleave(H // Hk, 1)
    qh = torch.where(anyrow[..., None], q.transpose(1, 2), 0.0)
    s = scale * qh @ kh.transpose(-1, -2)
    s = torch.where(seen, s, -math.inf)
    lse = torch.logsumexp(s, -1) if Tk else torch.full((B, H, Tq), -math.inf, dtype=torch.float64)
    p = torch.where(seen, torch.exp(s - torch.where(some, lse, 0.0)[..., None]), 0.0)
    o = p @ vh
    # scores: D products summed in float32, then their scaling; e_p is the relative error of a probability
    sizes = scale * (qh.abs() @ kh.abs().transpose(-1, -2))
    e_s = torch.where(seen, (D + 4) * U32 * sizes, 0.0)
    worst = e_s.amax(-1, keepdim=True) if Tk else torch.zeros((B, H, Tq, 1), dtype=torch.float64)
    lse0 = torch.where(some, lse, 0.0)[..., None]
    span = torch.where(seen, s.abs(), 0.0).amax(-1, keepdim=True) if Tk else worst
    e_p = e_s + worst + 4 * U32 * (span + lse0.abs()) + 16 * U32 + Tk * U32
    pv = p @ vh.abs()
    e_o = ((u + e_p) * p) @ vh.abs() + Tk * U32 * pv
    out = {"o": o.transpose(1, 2), "lse": lse,
           "e_o": (e_o + ROUND[dtype] * o.abs() + TINY[dtype]).transpose(1, 2),
           "e_lse": (worst + 4 * U32 * (span + lse0.abs()))[..., 0] + (16 + Tk) * U32}
    if do is not None:
        doh = torch.where(anyrow[..., None], do.transpose(1, 2), 0.0)
        dp = doh @ vh.transpose(-1, -2)
        delta = (doh * o).sum(-1, keepdim=True)
        ds = scale * p * (dp - delta)
        e_delta = (doh.abs() * (e_o + ROUND[dtype] * o.abs() + TINY[dtype])).sum(-1, keepdim=True) \
            + D * U32 * (doh * o).abs().sum(-1, keepdim=True)
        e_dp = D * U32 * (doh.abs() @ vh.abs().transpose(-1, -2))
        e_ds = scale * p * ((e_p + 8 * U32) * (dp.abs() + delta.abs()) + e_dp + e_delta) + u * ds.abs()
        group = lambda t: t.reshape(B, Hk, H // Hk, Tk, D).sum(2).transpose(1, 2)  # noqa: E731
        tr = lambda t: t.transpose(-1, -2)  # noqa: E731
        n = Tq * (H // Hk)
        out["dq"] = (ds @ kh).transpose(1, 2)
        out["e_dq"] = ((e_ds + Tk * U32 * ds.abs()) @ kh.abs()).transpose(1, 2) + ROUND[dtype] * out["dq"].abs()
        out["dk"] = group(tr(ds) @ qh)
        out["e_dk"] = group(tr(e_ds + n * U32 * ds.abs()) @ qh.abs()) + ROUND[dtype] * out["dk"].abs()
        out["dv"] = group(tr(p) @ doh)
        out["e_dv"] = group(tr((u + e_p + n * U32) * p) @ doh.abs()) + ROUND[dtype] * out["dv"].abs()
        for name in ("dq", "dk", "dv"):
            out["e_" + name] = out["e_" + name] + TINY[dtype]
    return out
