"""Splats predicted from an image by a small decoder, trained through the rasterizer.

The image's 8 x 8 patches become tokens (a linear layer, group norm with SiLU), learned splat queries on a grid attend to
them (rotary positions with two axes on queries and keys, cross attention), and a linear head turns each query's result
into one Gaussian, which is projected, binned and rendered; the L1 + SSIM loss runs back the same way and one fused Adam
step updates every weight, or, with --optimiser muon, Adam the norm and the queries and orthogonalised momentum the
matrices. Everything but the linear layers (torch matrix products) is the library's.

    python examples/splats_from_image.py [--steps 60] [--optimiser muon]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from differentiable_gaussian_splatting_amd import gsr  # noqa: E402

SIZE, PATCH, CHANNELS, GROUPS, HEADS, SIDE = 128, 8, 64, 8, 4, 24
PAIRS = (CHANNELS // HEADS // 4,) * 2  # half of a head's pairs follow y, half x


def weights(seed=0, device="cuda"):
    """The trained tensors: patch embedding, key and value maps, head, norm scale and shift, splat queries."""
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, scale):
        return (scale * torch.randn(shape, generator=g)).to(device)

    return {"embed": normal(PATCH * PATCH * 3, CHANNELS, scale=(PATCH * PATCH * 3) ** -0.5),
            "key": normal(CHANNELS, CHANNELS, scale=CHANNELS ** -0.5),
            "value": normal(CHANNELS, CHANNELS, scale=CHANNELS ** -0.5),
            "head": normal(CHANNELS, 10, scale=0.1),
            "gamma": torch.ones(CHANNELS, device=device), "beta": torch.zeros(CHANNELS, device=device),
            "queries": normal(SIDE * SIDE, CHANNELS, scale=0.5)}


def patches_of(image):
    """[H, W, 3] -> [tokens, values of an 8 x 8 patch]."""
    h, w = image.shape[0] // PATCH, image.shape[1] // PATCH
    return image.reshape(h, PATCH, w, PATCH, 3).transpose(1, 2).reshape(h * w, PATCH * PATCH * 3).contiguous()


def grid(side, cells, device="cuda"):
    """(y, x) of side x side points spread over `cells` units, as positions [1, side^2, 2]."""
    at = (torch.arange(side, device=device, dtype=torch.float32) + 0.5) * (cells / side)
    return torch.stack(torch.meshgrid(at, at, indexing="ij"), -1).reshape(1, side * side, 2).contiguous()


def decoder_forward(ctx, w, patches, pos_q, pos_k):
    """Returns the head's output [queries, 10] and what the backward needs."""
    tokens = patches.shape[0]
    x = (patches @ w["embed"]).reshape(1, tokens, CHANNELS)
    h, stats = gsr.gsr_group_norm_forward(ctx, x, w["gamma"], w["beta"], GROUPS, 1e-5, gsr.GSR_ACT_SILU)
    k = (h[0] @ w["key"]).reshape(1, tokens, HEADS, -1)
    v = (h[0] @ w["value"]).reshape(1, tokens, HEADS, -1)
    q = w["queries"].reshape(1, -1, HEADS, CHANNELS // HEADS)
    q = gsr.gsr_rotary_forward(ctx, q, pos_q, PAIRS, 100.0)
    k = gsr.gsr_rotary_forward(ctx, k, pos_k, PAIRS, 100.0)
    o, lse = gsr.gsr_cross_attention_forward(ctx, q, k, v)
    return o.reshape(-1, CHANNELS) @ w["head"], (patches, x, stats, h, q, k, v, o, lse)


def decoder_backward(ctx, w, saved, pos_q, pos_k, dout):
    """The gradient of every weight for the gradient `dout` of the head's output."""
    patches, x, stats, h, q, k, v, o, lse = saved
    g = {"head": o.reshape(-1, CHANNELS).T @ dout}
    do = (dout @ w["head"].T).reshape(o.shape)
    dq, dk, dv = gsr.gsr_cross_attention_backward(ctx, q, k, v, o, lse, do)
    dq = gsr.gsr_rotary_backward(ctx, dq, pos_q, PAIRS, 100.0)
    dk = gsr.gsr_rotary_backward(ctx, dk, pos_k, PAIRS, 100.0).reshape(-1, CHANNELS)
    dv = dv.reshape(-1, CHANNELS)
    g["queries"] = dq.reshape(-1, CHANNELS)
    g["key"], g["value"] = h[0].T @ dk, h[0].T @ dv
    dh = (dk @ w["key"].T + dv @ w["value"].T).reshape(x.shape)
    dx, g["gamma"], g["beta"] = gsr.gsr_group_norm_backward(ctx, x, w["gamma"], w["beta"], GROUPS, stats, dh,
                                                            gsr.GSR_ACT_SILU)
    g["embed"] = patches.T @ dx[0]
    return g


def gaussians(out):
    """One Gaussian per query: offsets from a grid in the plane z = 0, scales, opacity and colour."""
    n = out.shape[0]
    at = grid(SIDE, 4.0, out.device)[0] - 2.0
    means = torch.zeros((n, 3), device=out.device)
    means[:, 0], means[:, 1] = at[:, 1], at[:, 0]
    means += 0.1 * out[:, 0:3]
    quats = torch.zeros((n, 4), device=out.device)
    quats[:, 0] = 1
    sh = torch.zeros((n, 16, 3), device=out.device)
    sh[:, 0] = out[:, 7:10]
    return means, (-2.5 + out[:, 3:6]).contiguous(), quats, out[:, 6].contiguous(), sh


MATRICES = ("embed", "key", "value", "head")


def update(ctx, w, grads, state, step, optimiser):
    """One step of the optimiser on every weight; `state` holds two buffers a weight (a momentum is the first)."""
    by_adam = [k for k in w if optimiser == "adam" or k not in MATRICES]
    groups = [(w[k], grads[k].contiguous(), *state[k], 2e-3) for k in by_adam]
    gsr.gsr_adam_step(ctx, groups, 0.9, 0.999, 1e-8, 1 - 0.9 ** step, 1 - 0.999 ** step)
    for k in w:
        if k not in by_adam:  # an update whose elements are about as large as Adam's, whatever the matrix's shape
            gsr.gsr_muon_step(ctx, w[k], grads[k].contiguous(), state[k][0], 2e-3 * max(w[k].shape) ** 0.5)


def train(steps=60, seed=0, say=print, optimiser="adam"):
    """Fits the decoder to one synthetic image; returns the losses."""
    ctx = gsr.Context(0)
    yx = grid(SIZE, 1.0)[0].reshape(SIZE, SIZE, 2)
    target = torch.stack([yx[..., 0], 0.5 + 0.5 * torch.sin(9 * yx[..., 1]),
                          ((yx - 0.5).norm(dim=-1) < 0.3).float()], -1).contiguous()
    w = weights(seed)
    state = {k: (torch.zeros_like(t), torch.zeros_like(t)) for k, t in w.items()}
    patches = patches_of(target)
    cells = SIZE // PATCH
    pos_q, pos_k = grid(SIDE, cells), grid(cells, cells)
    cam = gsr.camera(torch.eye(3), [0, 0, 4], SIZE, SIZE, SIZE / 2, SIZE / 2)
    losses = []
    for step in range(1, steps + 1):
        out, saved = decoder_forward(ctx, w, patches, pos_q, pos_k)
        params = gaussians(out)
        splats, depths = gsr.gsr_project_forward(ctx, cam, *params)
        bins = gsr.gsr_bin(ctx, splats, depths, SIZE, SIZE)
        image, final_t, last = gsr.gsr_render_forward(ctx, splats, bins, SIZE, SIZE)
        v_out, loss = gsr.gsr_loss_l1_ssim(ctx, image, target)
        dsplats = gsr.gsr_render_backward(ctx, splats, bins, SIZE, SIZE, image, final_t, last, v_out)
        dmeans, dscales, _, dopacity, dsh = gsr.gsr_project_backward(ctx, cam, *params, dsplats)
        dout = torch.cat([0.1 * dmeans, dscales, dopacity[:, None], dsh[:, 0]], -1)
        grads = decoder_backward(ctx, w, saved, pos_q, pos_k, dout)
        update(ctx, w, grads, state, step, optimiser)
        losses.append(float(loss[0]))
        if step == 1 or step % 20 == 0:
            say(f"step {step}: loss {losses[-1]:.4f}", flush=True)
    ctx.close()
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--optimiser", choices=("adam", "muon"), default="adam")
    args = ap.parse_args()
    train(args.steps, optimiser=args.optimiser)
