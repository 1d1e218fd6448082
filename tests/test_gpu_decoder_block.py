"""A block of a decoder as it is trained: layer norm, cross attention to image tokens, layer norm, a feed-forward layer,
their backward pass, and the optimiser's step on every weight (orthogonalised momentum for the matrices, Adam for the
norms), twice; and the example's training with that optimiser.

Bar of the gradients: float32 against float64 through five matrix products, two norms and an attention, each rounding near
2^-24 of its terms with sums of at most a few hundred of them; 1e-4 of a gradient's norm is several hundred times that."""
import importlib.util
import os

import pytest
import torch

from featurehelp import normal
from gpuhelp import banner
from oracle import features as of

pytestmark = pytest.mark.gpu
T, S, C, H = 70, 130, 64, 4
QUINTIC = [(3.4445, -4.7750, 2.0315)] * 5


def weights():
    w = {k: normal(i, s, scale=s[0] ** -0.5) for i, (k, s) in enumerate(
        {"q": (C, C), "k": (C, C), "v": (C, C), "o": (C, C), "up": (C, 4 * C), "down": (4 * C, C)}.items())}
    for i in (1, 2):
        w[f"g{i}"], w[f"b{i}"] = 1 + 0.2 * normal(10 + i, (C,)), 0.2 * normal(20 + i, (C,))
    return w


def forward(ctx, w, x, image):
    from differentiable_gaussian_splatting_amd import gsr
    heads = lambda t: t.reshape(1, -1, H, C // H)  # noqa: E731
    a, sa = gsr.gsr_layer_norm_forward(ctx, x, w["g1"], w["b1"])
    q, k, v = heads(a @ w["q"]), heads(image @ w["k"]), heads(image @ w["v"])
    o, lse = gsr.gsr_cross_attention_forward(ctx, q, k, v)
    h = x + o.reshape(-1, C) @ w["o"]
    c, sc = gsr.gsr_layer_norm_forward(ctx, h, w["g2"], w["b2"])
    u = c @ w["up"]
    z = torch.nn.functional.silu(u)
    return h + z @ w["down"], (a, sa, q, k, v, o, lse, h, c, sc, u, z)


def backward(ctx, w, x, image, saved, dy):
    from differentiable_gaussian_splatting_amd import gsr
    a, sa, q, k, v, o, lse, h, c, sc, u, z = saved
    t = lambda m: m.T.contiguous()  # noqa: E731
    g = {"down": t(z) @ dy}
    s = torch.sigmoid(u)
    du = (dy @ t(w["down"])) * s * (1 + u * (1 - s))
    g["up"] = t(c) @ du
    dh, g["g2"], g["b2"] = gsr.gsr_layer_norm_backward(ctx, h, w["g2"], sc, du @ t(w["up"]))
    dh = dh + dy
    g["o"] = t(o.reshape(-1, C)) @ dh
    dq, dk, dv = gsr.gsr_cross_attention_backward(ctx, q, k, v, o, lse, (dh @ t(w["o"])).reshape(o.shape))
    dq, dk, dv = (m.reshape(-1, C) for m in (dq, dk, dv))
    g["q"], g["k"], g["v"] = t(a) @ dq, t(image) @ dk, t(image) @ dv
    dx, g["g1"], g["b1"] = gsr.gsr_layer_norm_backward(ctx, x, w["g1"], sa, dq @ t(w["q"]))
    return dx + dh, g


def reference(w, x, image):
    norm = torch.nn.functional.layer_norm
    heads = lambda t: t.reshape(-1, H, C // H).transpose(0, 1)  # noqa: E731
    a = norm(x, (C,), w["g1"], w["b1"])
    q, k, v = heads(a @ w["q"]), heads(image @ w["k"]), heads(image @ w["v"])
    p = torch.softmax(q @ k.transpose(1, 2) * (C // H) ** -0.5, -1)
    h = x + (p @ v).transpose(0, 1).reshape(-1, C) @ w["o"]
    return h + torch.nn.functional.silu(norm(h, (C,), w["g2"], w["b2"]) @ w["up"]) @ w["down"]


def test_a_block_trains():
    from differentiable_gaussian_splatting_amd import gsr
    banner("decoder block: two training steps")
    ctx = gsr.Context(0)
    try:
        w = {k: t.cuda() for k, t in weights().items()}
        state = {k: (torch.zeros_like(t), torch.zeros_like(t)) for k, t in w.items()}
        x, image, dy = normal(31, (T, C)).cuda(), normal(32, (S, C)).cuda(), normal(33, (T, C)).cuda()
        lr, mu, decay = 0.02, 0.95, 0.99
        for step in (1, 2):
            y, saved = forward(ctx, w, x, image)
            dx, g = backward(ctx, w, x, image, saved, dy)
            d = {k: t.cpu().double().requires_grad_(True) for k, t in (("x", x), *w.items())}
            ref = reference(d, d["x"], image.cpu().double())
            assert float((y.cpu().double() - ref.detach()).norm() / ref.detach().norm()) < 1e-5
            for name, want in zip(d, torch.autograd.grad(ref, list(d.values()), dy.cpu().double())):
                err = float(((dx if name == "x" else g[name]).cpu().double() - want).norm() / want.norm())
                print(f"  step {step} {name}: {err:.2e}")
                assert err < 1e-4, name
            before = {k: (t.cpu().double(), state[k][0].cpu().double()) for k, t in w.items()}
            gsr.gsr_adam_step(ctx, [(w[k], g[k], *state[k], 1e-3) for k in w if w[k].dim() == 1], 0.9, 0.999, 1e-8,
                              1 - 0.9 ** step, 1 - 0.999 ** step)
            for k in w:
                if w[k].dim() == 2:
                    gsr.gsr_muon_step(ctx, w[k], g[k], state[k][0], lr, mu, True, decay)
                    m = mu * before[k][1] + g[k].cpu().double()
                    u = g[k].cpu().double() + mu * m
                    o = of.newton_schulz(u, QUINTIC, 1e-7)
                    # u's and the products' roundings, 2^-22 of the largest singular value, grow at most by the steps'
                    # slope at 0, 3.4445^5 = 485, in each of the at most 64 directions
                    bound = lr * 485 * 2.0 ** -22 * 64 ** 0.5 + 2.0 ** -22 * float(before[k][0].norm())
                    assert float((w[k].cpu().double() - (decay * before[k][0] - lr * o)).norm()) < bound, k
    finally:
        ctx.close()


def test_the_example_runs_with_it():
    banner("splat decoder trained by orthogonalised momentum")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("splats_from_image", os.path.join(root, "examples",
                                                                                   "splats_from_image.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses = m.train(5, optimiser="muon")
    assert len(losses) == 5 and all(x == x for x in losses)
