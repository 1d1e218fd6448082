"""Timed cases of the operators that train a decoder of splats beyond its attention: layer norm over token features,
forward and backward, the orthogonalisation of a matrix update by Newton-Schulz products, and the optimiser step that
applies it to a decoder's weight matrices.

With own = False every operator is computed in its plain form, elementary torch operations in 32 bits; with own = True
by the library's entry points. Numbers of tokens follow the rasterizer's own 800 x 800 image (one token per 16 x 16 tile
is 50 x 50 = 2,500, one per 8 x 8 block 100 x 100 = 10,000); widths and weight shapes are those of small and large
decoders, the smallest those of examples/splats_from_image.py.
"""
from __future__ import annotations

import math

import torch

own = False

_DTYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
_COEFFICIENTS = (3.4445, -4.7750, 2.0315)
_STEPS, _EPS = 5, 1e-7
_MOMENTUM, _LR, _DECAY = 0.95, 0.02, 0.998
_ctx = None


def listed():
    return [
        # Layer norm. One splat query added to a served reconstruction, where the launch counts; a training step's
        # smallest, odd map (a 17 x 19 crop of three views, 90 channels: rows that are no multiple of 16 bytes); the
        # tokens of four views, forward only (serving); training in float32 with one token per tile; training on every
        # token of four views, where the weight's gradient sums 40,000 rows.
        _ln("ln_forward_one_token_bf16", "forward", 1, 1, 1024, "bfloat16"),
        _ln("ln_train_small_odd_f16", "train", 3, 323, 90, "float16"),
        _ln("ln_forward_views_bf16", "forward", 4, 10000, 1024, "bfloat16"),
        _ln("ln_train_tiles_f32", "train", 4, 2500, 640, "float32"),
        _ln("ln_train_views_bf16", "train", 4, 10000, 1024, "bfloat16"),
        # Orthogonalised updates. The example decoder's key and value maps; two odd, wide matrices (a narrow head); the
        # square projections of twelve layers, stacked; one tall matrix in float32.
        _orth("orthogonalize_small_f32", 2, 64, 64, "float32"),
        _orth("orthogonalize_odd_f16", 2, 333, 1111, "float16"),
        _orth("orthogonalize_stack_bf16", 12, 1024, 1024, "bfloat16"),
        _orth("orthogonalize_tall_f32", 1, 4096, 1024, "float32"),
        # Optimiser steps. The example decoder's patch embedding; the feed-forward weights of eight layers with bfloat16
        # gradients; one large square matrix with float32 gradients.
        _muon("muon_embedding_f32", 1, 192, 64, "float32"),
        _muon("muon_feed_forward_bf16", 8, 1024, 4096, "bfloat16"),
        _muon("muon_large_f32", 1, 4096, 4096, "float32"),
    ]


def _ln(name, way, batch, tokens, channels, dtype):
    return {"name": name, "op": "layer_norm", "way": way, "batch": batch, "tokens": tokens, "channels": channels,
            "dtype": dtype}


def _orth(name, batch, rows, cols, dtype):
    return {"name": name, "op": "orthogonalize", "batch": batch, "rows": rows, "cols": cols, "dtype": dtype}


def _muon(name, batch, rows, cols, dtype, nesterov=True):
    return {"name": name, "op": "muon", "batch": batch, "rows": rows, "cols": cols, "dtype": dtype,
            "nesterov": nesterov}


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    """One more case of the listed ranges: sizes spread over their logarithm, odd ones among them."""
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    dtype = rng.choice(["float32", "float16", "bfloat16"])
    op = rng.choice(["layer_norm", "orthogonalize", "muon"])
    while True:
        if op == "layer_norm":
            way = rng.choice(["forward", "train"])
            channels = rng.choice([spread(8, 4096), 8 * spread(1, 512)])
            case = _ln("", way, rng.randint(1, 4), spread(1, 10000), channels, dtype)
            top = "ln_forward_views_bf16" if way == "forward" else "ln_train_views_bf16"
        else:
            rows, cols = (rng.choice([spread(10, 4096), 16 * spread(1, 256)]) for _ in range(2))
            batch = rng.choice([1, 1, 2, spread(1, 16)])
            if op == "orthogonalize":
                case, top = _orth("", batch, rows, cols, dtype), "orthogonalize_tall_f32"
            else:
                case, top = _muon("", batch, rows, cols, dtype, rng.choice([True, False])), "muon_large_f32"
        if _cost(case) <= _cost(next(c for c in listed() if c["name"] == top)):
            del case["name"]
            return case


def work(case):
    size = 4 if case["dtype"] == "float32" else 2
    if case["op"] == "layer_norm":
        rows, c = case["batch"] * case["tokens"], case["channels"]
        # forward reads x and writes y; a training step also reads x and dy again and writes dx
        if case["way"] == "forward":
            return {"bytes": rows * (2 * c * size + 8) + 8 * c, "flops": 8 * rows * c}
        return {"bytes": rows * (5 * c * size + 16) + 20 * c, "flops": 22 * rows * c}
    b, m, n = case["batch"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
    # a step's products: X X^T and A^2, symmetric, of which half the elements are computed, and B X
    flops = b * _STEPS * (m * m * n + m * m * m + 2 * m * m * n)
    if case["op"] == "orthogonalize":
        return {"bytes": 2 * b * m * n * size, "flops": flops}
    # the gradient read, parameter and momentum read and written
    return {"bytes": b * m * n * (size + 16), "flops": flops}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype = _DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    s = {"case": dict(case)}
    if case["op"] == "layer_norm":
        b, t, c = case["batch"], case["tokens"], case["channels"]
        # a residual stream: each channel with a centre and a scale of its own, each token with a length of its own
        s["x"] = ((normal(b, t, c) * (0.5 + normal(c).abs()) + normal(c)) * torch.exp(0.5 * normal(b, t, 1))).to(dtype)
        s["gamma"] = 1 + 0.1 * normal(c)
        s["beta"] = 0.1 * normal(c)
        if case["way"] == "train":
            s["dy"] = normal(b, t, c).to(dtype)
        return s
    b, m, n = case["batch"], case["rows"], case["cols"]

    def gradient():
        """A few strong directions over noise, of a loss gradient's small magnitude."""
        k = min(m, n, 8)
        strong = torch.bmm(normal(b, m, k), normal(b, k, n).contiguous()) / math.sqrt(k)
        return 1e-3 * (strong + normal(b, m, n))

    s["grad"] = gradient().to(dtype)
    if case["op"] == "muon":
        s["param"] = normal(b, m, n) * n ** -0.5
        s["momentum"] = 5 * gradient()
        s["lr"] = _LR * 0.2 * math.sqrt(max(m, n))  # an update whose elements are of one size whatever the shape
    return s


def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    if case["op"] == "layer_norm":
        return _plain_layer_norm(case, state)
    if case["op"] == "orthogonalize":
        return _plain_orthogonalize(state["grad"].float()).to(state["grad"].dtype)
    return _plain_muon(case, state)


def _own(case, s):
    global _ctx
    from differentiable_gaussian_splatting_amd import gsr
    if _ctx is None:
        _ctx = gsr.Context(0)
    if case["op"] == "layer_norm":
        y, stats = gsr.gsr_layer_norm_forward(_ctx, s["x"], s["gamma"], s["beta"], 1e-5)
        out = {"y": y, "stats": stats}
        if case["way"] == "train":
            out["dx"], out["dgamma"], out["dbeta"] = gsr.gsr_layer_norm_backward(_ctx, s["x"], s["gamma"], stats, s["dy"])
        return out
    if case["op"] == "orthogonalize":
        return gsr.gsr_orthogonalize(_ctx, s["grad"], _STEPS, _COEFFICIENTS, _EPS)
    gsr.gsr_muon_step(_ctx, s["param"], s["grad"], s["momentum"], s["lr"], _MOMENTUM, case["nesterov"], _DECAY, _STEPS,
                      _COEFFICIENTS, _EPS)
    return {"param": s["param"], "momentum": s["momentum"]}


def _plain_layer_norm(case, s):
    x = s["x"].float()
    mean = x.mean(-1, keepdim=True)
    centred = x - mean
    rstd = (centred.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
    xh = centred * rstd
    out = {"y": (xh * s["gamma"] + s["beta"]).to(s["x"].dtype), "stats": torch.cat([mean, rstd], -1)}
    if case["way"] == "train":
        dy = s["dy"].float()
        dh = dy * s["gamma"]
        dx = rstd * (dh - dh.mean(-1, keepdim=True) - xh * (dh * xh).mean(-1, keepdim=True))
        out["dx"] = dx.to(s["x"].dtype)
        out["dgamma"] = (dy * xh).sum((0, 1))
        out["dbeta"] = dy.sum((0, 1))
    return out


def _plain_orthogonalize(g):
    """X = g / (|g| + eps), then X <- a X + (b A + c A^2) X with A = X X^T, for each matrix of g, float32 [b, m, n]."""
    a, b, c = _COEFFICIENTS
    tall = g.shape[1] > g.shape[2]
    x = g.transpose(1, 2).contiguous() if tall else g
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + _EPS)
    for _ in range(_STEPS):
        gram = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * gram + c * torch.bmm(gram, gram), x)
    return x.transpose(1, 2).contiguous() if tall else x


def _plain_muon(case, s):
    g = s["grad"].float()
    s["momentum"].mul_(_MOMENTUM).add_(g)
    update = g + _MOMENTUM * s["momentum"] if case["nesterov"] else s["momentum"]
    s["param"].mul_(_DECAY).sub_(s["lr"] * _plain_orthogonalize(update))
    return {"param": s["param"], "momentum": s["momentum"]}


def exact(case, seed):
    """The operators' definitions in 64 bits; layer norm's gradients by automatic differentiation."""
    s = prepare(case, seed)
    if case["op"] == "layer_norm":
        x, gamma, beta = (s[k].double().requires_grad_(True) for k in ("x", "gamma", "beta"))
        var, mean = torch.var_mean(x.detach(), -1, correction=0, keepdim=True)
        y = torch.nn.functional.layer_norm(x, x.shape[-1:], gamma, beta, 1e-5)
        out = {"y": y.detach(), "stats": torch.cat([mean, 1 / torch.sqrt(var + 1e-5)], -1)}
        if case["way"] == "train":
            out["dx"], out["dgamma"], out["dbeta"] = torch.autograd.grad(y, (x, gamma, beta), s["dy"].double())
        return out
    grad = s["grad"].double()
    if case["op"] == "orthogonalize":
        return torch.stack([_polar_like(g) for g in grad])
    momentum = _MOMENTUM * s["momentum"].double() + grad
    update = torch.add(grad, momentum, alpha=_MOMENTUM) if case["nesterov"] else momentum
    param = s["param"].double() * _DECAY - s["lr"] * torch.stack([_polar_like(u) for u in update])
    return {"param": param, "momentum": momentum}


def _polar_like(g):
    """The odd polynomial x (a + b x^2 + c x^4), applied to the singular values of g / (|g| + eps) five times over, by
    products on the smaller side, innermost first."""
    if g.shape[0] > g.shape[1]:
        return _polar_like(g.T.contiguous()).T
    a, b, c = _COEFFICIENTS
    x = g / (torch.linalg.matrix_norm(g) + _EPS)
    for _ in range(_STEPS):
        xt = x.T.contiguous()
        if x.shape[1] > 2 * x.shape[0]:
            gram = x @ xt
            x = a * x + gram @ (b * x + c * (gram @ x))
        else:
            right = xt @ x
            x = a * x + (b * x + c * (x @ right)) @ right
    return x
