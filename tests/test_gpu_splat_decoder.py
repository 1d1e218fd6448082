"""The example decoder (examples/splats_from_image.py): the chained operators' weight gradients against automatic
differentiation of the same decoder in float64, and a training run through the rasterizer.

Bar of the gradients: float32 against float64 through three matrix products, a norm and an attention, each rounding near
2^-24 of its terms with sums of at most a few hundred of them; 1e-4 of a gradient's norm is several hundred times that."""
import importlib.util
import os

import pytest
import torch

from gpuhelp import banner

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("splats_from_image",
                                                  os.path.join(ROOT, "examples", "splats_from_image.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def turned(x, pos, pairs, base):
    f = torch.cat([base ** (-torch.arange(p, dtype=torch.float64) / p) for p in pairs])
    axis = [a for a, p in enumerate(pairs) for _ in range(p)]
    z = torch.view_as_complex(x.unflatten(-1, (-1, 2)).contiguous())
    return torch.view_as_real(z * torch.polar(torch.ones_like(pos[:, :, axis]), pos[:, :, axis] * f)[:, :, None]
                              ).flatten(-2)


def test_decoder_gradients():
    from differentiable_gaussian_splatting_amd import gsr
    ex = example()
    banner("splat decoder gradients")
    ctx = gsr.Context(0)
    try:
        w = ex.weights(3)
        w["gamma"] += 0.3 * torch.randn(ex.CHANNELS, generator=torch.Generator().manual_seed(1)).cuda()
        image = torch.rand((ex.SIZE, ex.SIZE, 3), generator=torch.Generator().manual_seed(2)).cuda()
        cells = ex.SIZE // ex.PATCH
        pos_q, pos_k, patches = ex.grid(ex.SIDE, cells), ex.grid(cells, cells), ex.patches_of(image)
        out, saved = ex.decoder_forward(ctx, w, patches, pos_q, pos_k)
        dout = torch.randn(out.shape, generator=torch.Generator().manual_seed(4)).cuda()
        got = ex.decoder_backward(ctx, w, saved, pos_q, pos_k, dout)
    finally:
        ctx.close()
    d = {k: t.cpu().double().requires_grad_(True) for k, t in w.items()}
    x = patches.cpu().double() @ d["embed"]
    h = torch.nn.functional.silu(torch.nn.functional.group_norm(x.T[None], ex.GROUPS, d["gamma"], d["beta"], 1e-5))[0].T
    heads = lambda t: t.reshape(1, -1, ex.HEADS, ex.CHANNELS // ex.HEADS)  # noqa: E731
    q = turned(heads(d["queries"]), pos_q.cpu().double(), ex.PAIRS, 100.0).transpose(1, 2)
    k = turned(heads(h @ d["key"]), pos_k.cpu().double(), ex.PAIRS, 100.0).transpose(1, 2)
    v = heads(h @ d["value"]).transpose(1, 2)
    p = torch.softmax(q @ k.transpose(-1, -2) * (ex.CHANNELS // ex.HEADS) ** -0.5, -1)
    ref = (p @ v).transpose(1, 2).reshape(-1, ex.CHANNELS) @ d["head"]
    assert float((out.cpu().double() - ref.detach()).norm() / ref.detach().norm()) < 1e-5
    for name, want in zip(d, torch.autograd.grad(ref, list(d.values()), dout.cpu().double())):
        err = float((got[name].cpu().double() - want).norm() / want.norm())
        print(f"  {name}: {err:.2e}")
        assert err < 1e-4, name


def test_training_lowers_the_loss():
    banner("splat decoder training")
    losses = example().train(40)
    assert all(x == x for x in losses) and losses[-1] < 0.6 * losses[0], losses


def test_kernel_times_of_the_operators():
    from differentiable_gaussian_splatting_amd import gsr
    ex = example()
    banner("kernel times of the feature operators")
    ctx = gsr.Context(0)
    try:
        gsr.gsr_set_option(ctx, gsr.GSR_OPT_KERNEL_TIMING, 8)
        w, cells = ex.weights(3), ex.SIZE // ex.PATCH
        pos_q, pos_k = ex.grid(ex.SIDE, cells), ex.grid(cells, cells)
        patches = ex.patches_of(torch.rand((ex.SIZE, ex.SIZE, 3)).cuda())
        out, saved = ex.decoder_forward(ctx, w, patches, pos_q, pos_k)
        ex.decoder_backward(ctx, w, saved, pos_q, pos_k, out)
        counts = {gsr.GSR_STAGE_GROUP_NORM_FORWARD: 1, gsr.GSR_STAGE_GROUP_NORM_BACKWARD: 1, gsr.GSR_STAGE_ROTARY: 4,
                  gsr.GSR_STAGE_ATTENTION_FORWARD: 1, gsr.GSR_STAGE_ATTENTION_BACKWARD: 1}
        for stage, n in counts.items():
            t = gsr.gsr_kernel_times(ctx, stage)
            assert len(t) == n and all(0 < x < 1000 for x in t), (stage, t)
    finally:
        ctx.close()
