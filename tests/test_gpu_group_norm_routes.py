"""GPU group norm on both of its routes: one launch that keeps a map in registers, and several launches with partial sums
in the arena. Element by element within the fp64 oracle's bounds.

Which route a forward takes is read off its scratch: one launch needs none, so it works under an arena limit of one byte,
and several launches fail there. A backward needs some on either; 8,193 pixels and more are beyond the registers of a
workgroup (1,024 threads of 8 vectors forward, 4 backward, a pixel each at least)."""
import pytest
import torch

from featurehelp import DTYPES, normal, within
from gpuhelp import banner
from oracle import features as of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    from differentiable_gaussian_splatting_amd import gsr
    c = gsr.Context(0)
    yield c
    c.close()


@pytest.fixture(scope="module")
def bare():
    """A context that may hold no scratch."""
    from differentiable_gaussian_splatting_amd import gsr
    c = gsr.Context(0)
    gsr.gsr_set_option(c, gsr.GSR_OPT_ARENA_LIMIT, 1)
    yield c
    c.close()


@pytest.mark.parametrize("size", [1000.37, 3e4])
@pytest.mark.parametrize("noise", [0.0, 1.0])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_outliers_where_a_thread_adds_many_pixels(ctx, bare, dtype, noise, size):
    """One outlying pixel at the start of each run that a thread adds: 2,048 images leave one run an image, channels past
    the threads of a workgroup one thread a channel, so a run has all 256 pixels. The images are one map seen 2,048 times."""
    from differentiable_gaussian_splatting_amd import gsr
    banner(f"group norm outliers over long runs {dtype} noise {noise} size {size}")
    t, n, p = DTYPES[dtype], 2048, 256
    c = 1028 if dtype == "f32" else 2056
    x = (noise * normal(1, (1, p, c)))
    x[0, 0] = size
    x = x.to(t)
    xd = x.cuda().expand(n, p, c)
    with pytest.raises(gsr.GsrError) as e:  # several launches
        gsr.gsr_group_norm_forward(bare, xd, None, None, 1)
    assert e.value.status == gsr.GSR_ENOMEM
    y, stats = gsr.gsr_group_norm_forward(ctx, xd, None, None, 1)
    r = of.group_norm(x.double(), None, None, 1, 1e-5, "none")
    assert torch.equal(stats, stats[:1].expand(n, 1, 2)) and torch.equal(y[-1], y[0])
    within(stats[:1, :, 0], r["mean"], r["e_mean"], "mean")
    within(stats[:1, :, 1], r["rstd"], r["e_rstd"], "rstd")
    within(y[:1], r["y"], r["e_y"] + of.ROUND[t] * r["y"].abs() + of.TINY[t], "y")
