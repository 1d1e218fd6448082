"""Timed cases of the operators that predict splats from images: group norm with an activation over channels-last
feature maps, rotary positions with several axes, and cross attention from splat queries to image tokens.

With own = False every operator is computed in its plain form, elementary torch operations in 32 bits; with own = True
by the library's entry points. Sizes follow the rasterizer's own 800 x 800 image: one token per 16 x 16 tile is 50 x 50
= 2,500 tokens, one per 8 x 8 block is 100 x 100 = 10,000.
"""
from __future__ import annotations

import math

import torch

own = False

_DTYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
_ctx = None


def listed():
    return [
        # Group norm. A training step's smallest, odd map (a 17 x 19 crop, 90 channels: rows that are no multiple of 16
        # bytes), where launches count; a full-resolution 800 x 800 map of two views, forward only (serving); the
        # per-8x8-block maps of four views in training, 10 channels a group.
        _gn("gn_train_small_odd_f16", "train", 3, 17, 19, 90, 9, "float16"),
        _gn("gn_forward_800_bf16", "forward", 2, 800, 800, 64, 8, "bfloat16"),
        _gn("gn_train_100_f32", "train", 4, 100, 100, 320, 32, "float32"),
        # Rotary positions. One splat query (serving); the tokens of four views with (view, y, x) axes; the gradient of
        # queries whose head has an unrotated tail and rotates split halves.
        _rot("rotary_one_token_f32", "forward", 1, 1, 8, 64, "16,16", "interleaved", "float32"),
        _rot("rotary_views_bf16", "forward", 4, 10000, 16, 128, "16,24,24", "interleaved", "bfloat16"),
        _rot("rotary_backward_odd_f16", "backward", 2, 2501, 12, 80, "10,10,10", "halves", "float16"),
        # Cross attention. One query per scene added to a served reconstruction, ragged numbers of image tokens and
        # shared key heads; the same at its smallest, one short context; a prompt's worth of splat queries over a view's
        # 8x8 blocks; training with one query per tile; training in the library's own float32 with a visibility mask
        # (each query sees some views, some see none); training many queries on a short, odd context.
        _att("attn_one_query_bf16", "forward", 4, 1, 10000, 16, 4, 128, "bfloat16", ragged=True),
        _att("attn_one_query_small_f16", "forward", 1, 1, 257, 8, 8, 64, "float16"),
        _att("attn_forward_bf16", "forward", 1, 4096, 10000, 16, 16, 64, "bfloat16"),
        _att("attn_train_bf16", "train", 2, 2500, 2500, 8, 8, 128, "bfloat16"),
        _att("attn_train_masked_f32", "train", 2, 777, 1369, 6, 2, 48, "float32", views=4),
        _att("attn_train_short_f16", "train", 1, 10000, 77, 8, 8, 40, "float16"),
    ]


def _gn(name, way, n, h, w, c, groups, dtype):
    return {"name": name, "op": "group_norm", "way": way, "n": n, "h": h, "w": w, "c": c, "groups": groups, "dtype": dtype}


def _rot(name, way, batch, tokens, heads, dim, pairs, layout, dtype):
    return {"name": name, "op": "rotary", "way": way, "batch": batch, "tokens": tokens, "heads": heads, "dim": dim,
            "pairs": pairs, "layout": layout, "dtype": dtype}


def _att(name, way, batch, queries, keys, heads, kv_heads, dim, dtype, ragged=False, views=0):
    return {"name": name, "op": "attention", "way": way, "batch": batch, "queries": queries, "keys": keys,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "ragged": ragged, "views": views}


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    """One more case of the listed ranges: sizes spread over their logarithm, odd ones among them."""
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    dtype = rng.choice(["float32", "float16", "bfloat16"])
    op = rng.choice(["group_norm", "rotary", "attention", "attention"])
    while True:
        if op == "group_norm":
            groups = rng.choice([1, 4, 8, 9, 16, 32])
            case = _gn("", rng.choice(["forward", "train"]), rng.randint(1, 4), spread(8, 800), spread(8, 800),
                       groups * rng.choice([1, 2, 3, 4, 8, 10, 16]), groups, dtype)
            top = "gn_forward_800_bf16"
        elif op == "rotary":
            dim = rng.choice([32, 40, 64, 80, 96, 128])
            axes = rng.randint(1, 3)
            turned = dim // 2 - rng.choice([0, 0, 2, 5])
            pairs = [turned // axes] * (axes - 1)
            pairs.append(turned - sum(pairs))
            case = _rot("", rng.choice(["forward", "backward"]), rng.randint(1, 4), spread(1, 10000),
                        rng.choice([1, 6, 8, 12, 16]), dim, ",".join(map(str, pairs)),
                        rng.choice(["interleaved", "halves"]), dtype)
            top = "rotary_views_bf16"
        else:
            kv = rng.choice([1, 2, 4, 8])
            way = rng.choice(["forward", "train"])
            ragged, views = rng.choice([(False, 0), (True, 0), (False, 4), (False, 0)])
            case = _att("", way, rng.randint(1, 4), spread(1, 10000), spread(16, 10000), kv * rng.choice([1, 2, 4]), kv,
                        rng.choice([16, 24, 32, 40, 48, 64, 72, 80, 96, 128]), dtype, ragged, views)
            top = "attn_forward_bf16" if way == "forward" else "attn_train_bf16"
            # the plain form's scores, several of them in 32 bits, have to fit beside three states
            if case["batch"] * case["heads"] * case["queries"] * case["keys"] > 7e8:
                continue
        if _cost(case) <= _cost(next(c for c in listed() if c["name"] == top)):
            del case["name"]
            return case


def _lengths(case):
    """The number of valid keys of each batch entry: all of them, or a ragged spread down to about a third."""
    b, t = case["batch"], case["keys"]
    return [max(1, t - (i * 2 * t) // (3 * b)) for i in range(b)] if case["ragged"] else [t] * b


def work(case):
    size = 4 if case["dtype"] == "float32" else 2
    if case["op"] == "group_norm":
        e = case["n"] * case["h"] * case["w"] * case["c"]
        # forward reads x and writes y; a training step also reads x and dy again and writes dx
        return {"bytes": e * size * (2 if case["way"] == "forward" else 5) + 16 * case["c"],
                "flops": e * (10 if case["way"] == "forward" else 30)}
    if case["op"] == "rotary":
        tokens = case["batch"] * case["tokens"]
        axes = len(case["pairs"].split(","))
        return {"bytes": 2 * tokens * case["heads"] * case["dim"] * size + 4 * tokens * axes,
                "flops": 3 * tokens * case["heads"] * case["dim"]}
    q = case["batch"] * case["queries"] * case["heads"] * case["dim"] * size
    kv = 2 * sum(_lengths(case)) * case["kv_heads"] * case["dim"] * size
    rows = 4 * case["batch"] * case["queries"] * case["heads"]
    mask = case["batch"] * case["queries"] * case["keys"] if case["views"] else 0
    # a query's views differ from its neighbour's, so masked pairs are counted too: no block of them falls away
    pairs = case["queries"] * case["heads"] * sum(_lengths(case)) * case["dim"]
    if case["way"] == "forward":
        return {"bytes": 2 * q + kv + rows + mask, "flops": 4 * pairs}
    # forward, then: q, k, v, o, do, lse in, dq, dk, dv out
    return {"bytes": 2 * q + kv + rows + mask + 4 * q + 2 * kv + rows + mask, "flops": 14 * pairs}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype = _DTYPES[case["dtype"]]

    def normal(*shape, t=dtype):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(t)

    s = {"case": dict(case)}
    if case["op"] == "group_norm":
        n, h, w, c = case["n"], case["h"], case["w"], case["c"]
        # a convolution's output: each channel with a mean and a scale of its own
        centre, scale = normal(c, t=torch.float32), 0.5 + normal(c, t=torch.float32).abs()
        s["x"] = (torch.randn((n, h, w, c), generator=g, device="cuda") * scale + centre).to(dtype)
        s["gamma"] = 1 + 0.1 * normal(c, t=torch.float32)
        s["beta"] = 0.1 * normal(c, t=torch.float32)
        if case["way"] == "train":
            s["dy"] = normal(n, h, w, c)
    elif case["op"] == "rotary":
        b, t = case["batch"], case["tokens"]
        s["x"] = normal(b, t, case["heads"], case["dim"])
        s["pairs"] = [int(p) for p in case["pairs"].split(",")]
        # the last axis is x and the one before it y, on a square grid with sub-token offsets; the first of three is
        # the view
        side = max(1, math.isqrt(t))
        at = torch.arange(t, device="cuda", dtype=torch.float32)
        grid = torch.stack([torch.zeros_like(at), torch.div(at, side, rounding_mode="floor"), at % side], -1)
        pos = grid.expand(b, t, 3).contiguous()
        pos[:, :, 0] = torch.arange(b, device="cuda", dtype=torch.float32)[:, None]
        pos[:, :, 1:] += torch.rand((b, t, 2), generator=g, device="cuda")
        s["positions"] = pos[:, :, 3 - len(s["pairs"]):].contiguous()
    else:
        b, tq, tk = case["batch"], case["queries"], case["keys"]
        s["q"] = normal(b, tq, case["heads"], case["dim"])
        s["k"] = normal(b, tk, case["kv_heads"], case["dim"])
        s["v"] = normal(b, tk, case["kv_heads"], case["dim"])
        s["scale"] = case["dim"] ** -0.5
        s["lengths"] = torch.tensor(_lengths(case), device="cuda", dtype=torch.int32) if case["ragged"] else None
        s["mask"] = None
        if case["views"]:
            # each query sees seven of ten views, and one query in fifty none
            seen = torch.rand((b, tq, case["views"]), generator=g, device="cuda") < 0.7
            seen &= torch.rand((b, tq, 1), generator=g, device="cuda") >= 0.02
            view = torch.arange(tk, device="cuda") * case["views"] // tk
            s["mask"] = seen[:, :, view][:, None].contiguous()  # [b, 1, tq, tk]
        if case["way"] == "train":
            s["do"] = normal(b, tq, case["heads"], case["dim"])
    return s


def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    return {"group_norm": _plain_group_norm, "rotary": _plain_rotary, "attention": _plain_attention}[case["op"]](case, state)


def _own(case, s):
    global _ctx
    from differentiable_gaussian_splatting_amd import gsr
    if _ctx is None:
        _ctx = gsr.Context(0)
    if case["op"] == "group_norm":
        y, stats = gsr.gsr_group_norm_forward(_ctx, s["x"], s["gamma"], s["beta"], case["groups"], 1e-5, gsr.GSR_ACT_SILU)
        out = {"y": y, "stats": stats}
        if case["way"] == "train":
            out["dx"], out["dgamma"], out["dbeta"] = gsr.gsr_group_norm_backward(
                _ctx, s["x"], s["gamma"], s["beta"], case["groups"], stats, s["dy"], gsr.GSR_ACT_SILU)
        return out
    if case["op"] == "rotary":
        layout = gsr.GSR_ROTARY_INTERLEAVED if case["layout"] == "interleaved" else gsr.GSR_ROTARY_HALVES
        fn = gsr.gsr_rotary_forward if case["way"] == "forward" else gsr.gsr_rotary_backward
        return fn(_ctx, s["x"], s["positions"], s["pairs"], 10000.0, layout)
    o, lse = gsr.gsr_cross_attention_forward(_ctx, s["q"], s["k"], s["v"], s["scale"], s["lengths"], s["mask"])
    out = {"o": o, "lse": lse}
    if case["way"] == "train":
        out["dq"], out["dk"], out["dv"] = gsr.gsr_cross_attention_backward(
            _ctx, s["q"], s["k"], s["v"], o, lse, s["do"], s["scale"], s["lengths"], s["mask"])
    return out


def _plain_group_norm(case, s):
    n, c, groups = case["n"], case["c"], case["groups"]
    x = s["x"].float().reshape(n, -1, groups, c // groups)
    gamma, beta = (s[k].reshape(groups, c // groups) for k in ("gamma", "beta"))
    mean = x.mean((1, 3), keepdim=True)
    rstd = ((x - mean).square().mean((1, 3), keepdim=True) + 1e-5).rsqrt()
    xh = (x - mean) * rstd
    z = xh * gamma + beta
    sg = 1 / (1 + torch.exp(-z))
    out = {"y": (z * sg).reshape(s["x"].shape).to(s["x"].dtype),
           "stats": torch.stack([mean, rstd], -1).reshape(n, groups, 2)}
    if case["way"] == "train":
        dz = s["dy"].float().reshape(x.shape) * sg * (1 + z * (1 - sg))
        out["dgamma"] = (dz * xh).sum((0, 1)).reshape(c)
        out["dbeta"] = dz.sum((0, 1)).reshape(c)
        dh = dz * gamma
        dx = rstd * (dh - dh.mean((1, 3), keepdim=True) - xh * (dh * xh).mean((1, 3), keepdim=True))
        out["dx"] = dx.reshape(s["x"].shape).to(s["x"].dtype)
    return out


def _plain_rotary(case, s):
    x, turned = s["x"].float(), 2 * sum(s["pairs"])
    at = s["positions"][..., None]
    angle = torch.cat([at[:, :, a] * 10000.0 ** (-torch.arange(p, device=x.device, dtype=torch.float32) / p)
                       for a, p in enumerate(s["pairs"])], -1)[:, :, None]
    if case["way"] == "backward":
        angle = -angle
    cos, sin = torch.cos(angle), torch.sin(angle)
    out = x.clone()
    if case["layout"] == "interleaved":
        at, to = slice(0, turned, 2), slice(1, turned, 2)
    else:
        at, to = slice(0, turned // 2), slice(turned // 2, turned)
    u, v = x[..., at], x[..., to]
    out[..., at] = u * cos - v * sin
    out[..., to] = u * sin + v * cos
    return out.to(s["x"].dtype)


def _plain_attention(case, s):
    b, tq, tk, dim = case["batch"], case["queries"], case["keys"], case["dim"]
    kv, share = case["kv_heads"], case["heads"] // case["kv_heads"]

    def heads_first(x, n):  # [b, t, h, d] -> [b * kv, share, t, d], float32; n query heads share a key head
        return x.float().transpose(1, 2).reshape(b * kv, n * x.shape[1], dim).contiguous()

    def tokens_first(x, t, like):
        return x.reshape(b, -1, t, dim).transpose(1, 2).contiguous().to(like.dtype)

    q, k, v = heads_first(s["q"], share), heads_first(s["k"], 1), heads_first(s["v"], 1)
    score = torch.bmm(q, k.transpose(1, 2).contiguous()).mul_(s["scale"])
    if s["lengths"] is not None or s["mask"] is not None:
        seen = torch.ones((b, 1, 1, tk), dtype=torch.bool, device=q.device)
        if s["lengths"] is not None:
            seen = torch.arange(tk, device=q.device) < s["lengths"][:, None, None, None]
        if s["mask"] is not None:
            seen = seen & s["mask"]
        score.view(b, -1, tq, tk).masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min(-1e30)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p /= total.clamp_min(1e-30)
    lse = top + torch.log(total)
    o = torch.bmm(p, v)
    out = {"o": tokens_first(o, tq, s["q"]), "lse": lse.reshape(b, -1, tq)}
    if case["way"] == "train":
        do = heads_first(s["do"], share)
        out["dv"] = tokens_first(torch.bmm(p.transpose(1, 2).contiguous(), do), tk, s["v"])
        dp = torch.bmm(do, v.transpose(1, 2).contiguous())
        ds = dp.sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(s["scale"])
        out["dq"] = tokens_first(torch.bmm(ds, k), tq, s["q"])
        out["dk"] = tokens_first(torch.bmm(ds.transpose(1, 2).contiguous(), q), tk, s["k"])
    return out


def exact(case, seed):
    """The operators' definitions in 64 bits; gradients by automatic differentiation of the definition."""
    s = prepare(case, seed)
    if case["op"] == "group_norm":
        x, gamma, beta = (s[k].double().requires_grad_(True) for k in ("x", "gamma", "beta"))
        first = x.movedim(-1, 1).flatten(2)  # [n, c, p]
        grouped = first.reshape(case["n"], case["groups"], -1)
        var, mean = torch.var_mean(grouped, -1, correction=0)
        y = torch.nn.functional.group_norm(first, case["groups"], gamma, beta, 1e-5)
        y = torch.nn.functional.silu(y).reshape(x.movedim(-1, 1).shape).movedim(1, -1)
        out = {"y": y.detach(), "stats": torch.stack([mean, 1 / torch.sqrt(var + 1e-5)], -1).detach()}
        if case["way"] == "train":
            out["dx"], out["dgamma"], out["dbeta"] = torch.autograd.grad(y, (x, gamma, beta), s["dy"].double())
        return out
    if case["op"] == "rotary":
        x, pairs = s["x"].double(), s["pairs"]
        angle = torch.cat([s["positions"][:, :, a, None].double()
                           / torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=x.device),
                                       torch.arange(p, device=x.device, dtype=torch.float64) / p)
                           for a, p in enumerate(pairs)], -1)
        turn = torch.polar(torch.ones_like(angle), angle if case["way"] == "forward" else -angle)[:, :, None, :]
        rest = x[..., 2 * sum(pairs):]
        both = x[..., :2 * sum(pairs)]
        if case["layout"] == "interleaved":
            z = torch.view_as_complex(both.unflatten(-1, (-1, 2)).contiguous()) * turn
            both = torch.view_as_real(z).flatten(-2)
        else:
            u, v = both.chunk(2, -1)
            z = torch.complex(u.contiguous(), v.contiguous()) * turn
            both = torch.cat([z.real, z.imag], -1)
        return torch.cat([both, rest], -1)
    train = case["way"] == "train"
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    out = {"o": torch.zeros_like(q), "lse": torch.full((q.shape[0], q.shape[2], q.shape[1]), -math.inf,
                                                       dtype=torch.float64, device=q.device)}
    if train:
        out |= {"dq": torch.zeros_like(q), "dk": torch.zeros_like(k), "dv": torch.zeros_like(v)}
    for b, n in enumerate(_lengths(case)):
        for h in range(case["heads"]):
            j = h * case["kv_heads"] // case["heads"]
            qh, kh, vh = (x.contiguous().requires_grad_(train) for x in (q[b, :, h], k[b, :n, j], v[b, :n, j]))
            score = qh @ kh.T * s["scale"]
            some = torch.ones(case["queries"], dtype=torch.bool, device=q.device)
            if s["mask"] is not None:
                seen = s["mask"][b, 0, :, :n]
                some = seen.any(-1)
                score = score.masked_fill(~seen & some[:, None], -math.inf)
            o = (torch.softmax(score, -1) @ vh) * some[:, None]
            out["o"][b, :, h] = o.detach()
            out["lse"][b, h] = torch.logsumexp(score.detach(), -1).masked_fill(~some, -math.inf)
            if train:
                dq, dk, dv = torch.autograd.grad(o, (qh, kh, vh), s["do"][b, :, h].double())
                out["dq"][b, :, h] = dq
                out["dk"][b, :n, j] += dk
                out["dv"][b, :n, j] += dv
    return out
