"""GPU group norm on both of its routes: one launch that keeps a map in registers, and several launches with partial sums
in the arena. Element by element within the fp64 oracle's bounds.

Which route a forward takes is read off its scratch: one launch needs none, so it works under an arena limit of one byte,
and several launches fail there. 8,193 pixels and more are beyond the registers of a workgroup (1,024 threads of 8 vectors
forward, 4 backward, a pixel each at least), so their backward takes several launches too."""
import ctypes

import pytest
import torch

from featurehelp import DTYPES, normal, within
from gpuhelp import banner
from oracle import features as of

pytestmark = pytest.mark.gpu
KIND = {"none": 0, "silu": 1, "relu": 2}
MANY = 8500  # pixels of a map that takes several launches


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


def one_launch(bare, x, groups):
    from differentiable_gaussian_splatting_amd import gsr
    try:
        gsr.gsr_group_norm_forward(bare, x.cuda(), None, None, groups)
        return True
    except gsr.GsrError as e:
        assert e.status == gsr.GSR_ENOMEM
        return False


def features(seed, n, p, c, dtype, centre=0.7):
    x = normal(seed, (n, p, c)) * (0.5 + normal(seed + 1, (c,)).abs()) + centre * normal(seed + 2, (c,))
    return x.to(dtype)


def both(ctx, x, gamma, beta, groups, kind, dy, eps=1e-5):
    from differentiable_gaussian_splatting_amd import gsr
    d = lambda t: None if t is None else t.cuda()  # noqa: E731
    y, stats = gsr.gsr_group_norm_forward(ctx, d(x), d(gamma), d(beta), groups, eps, KIND[kind])
    return (y, stats) + gsr.gsr_group_norm_backward(ctx, d(x), d(gamma), d(beta), groups, stats, d(dy), KIND[kind])


def check(got, x, gamma, beta, groups, kind, dy, eps=1e-5):
    r = of.group_norm(x.double(), None if gamma is None else gamma.double(), None if beta is None else beta.double(),
                      groups, eps, kind, dy.double())
    u, tiny = of.ROUND[x.dtype], of.TINY[x.dtype]
    y, stats, dx, dgamma, dbeta = got
    within(stats[..., 0], r["mean"], r["e_mean"], "mean")
    within(stats[..., 1], r["rstd"], r["e_rstd"], "rstd")
    for name, t in (("y", y), ("dx", dx)):
        within(t, r[name], r["e_" + name] + u * r[name].abs() + tiny, name)
    within(dgamma, r["dgamma"], r["e_dgamma"] + of.U32 * r["dgamma"].abs(), "dgamma")
    within(dbeta, r["dbeta"], r["e_dbeta"] + of.U32 * r["dbeta"].abs(), "dbeta")


@pytest.mark.parametrize("kind", ["none", "relu", "silu"])
@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_several_launches(ctx, bare, dtype, kind, affine):
    banner(f"group norm several launches {dtype} {kind} affine {affine}")
    t = DTYPES[dtype]
    x, dy = features(3, 2, MANY, 24, t), normal(4, (2, MANY, 24), t)
    gamma, beta = (normal(5, (24,)), normal(6, (24,))) if affine else (None, None)
    assert not one_launch(bare, x, 4)
    check(both(ctx, x, gamma, beta, 4, kind, dy), x, gamma, beta, 4, kind, dy)


# maps above 1 MB that registers hold: sets of several groups, 16-byte vectors; a last set of fewer groups; vectors across
# groups and past the last channel
WIDE = [(32, 784, 240, 30), (70, 120, 78, 13), (40, 300, 320, 32), (130, 50, 252, 9)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n,p,c,groups", WIDE, ids=str)
def test_one_launch_of_wide_vectors(ctx, bare, dtype, n, p, c, groups):
    banner(f"group norm one launch, wide {dtype} {n} x {p} x {c} in {groups}")
    t = DTYPES[dtype]
    x, dy = features(n, n, p, c, t), normal(4, (n, p, c), t)
    gamma, beta = 1 + 0.2 * normal(5, (c,)), normal(6, (c,))
    assert x.numel() * x.element_size() > 1 << 20 and one_launch(bare, x, groups)
    for kind in ("silu", "relu"):
        check(both(ctx, x, gamma, beta, groups, kind, dy), x, gamma, beta, groups, kind, dy)


def test_far_mean_and_outlier(ctx, bare):
    """A mean of a thousand deviations, and an outlying first value, through the partial statistics."""
    banner("group norm several launches, far mean, outlying first value")
    x, dy = 1000 + normal(1, (1, MANY, 16)), normal(2, (1, MANY, 16))
    assert not one_launch(bare, x, 2)
    check(both(ctx, x, None, None, 2, "none", dy), x, None, None, 2, "none", dy)
    x[0, 0, :] = 1e5
    check(both(ctx, x, None, None, 2, "none", dy), x, None, None, 2, "none", dy)


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


def test_constant_features(ctx, bare):
    from differentiable_gaussian_splatting_amd import gsr
    banner("group norm several launches of a constant")
    x = torch.full((2, MANY, 12), 3.25, device="cuda")
    assert not one_launch(bare, x, 3)
    y, stats = gsr.gsr_group_norm_forward(ctx, x, None, None, 3, 1e-5)
    assert (y == 0).all() and (stats[..., 0] == 3.25).all()
    assert torch.allclose(stats[..., 1].cpu(), torch.tensor(1e-5).rsqrt(), rtol=1e-6)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("n,p,c", [(2, MANY, 24), (64, 400, 96)], ids=str)
def test_a_bad_value_stays_in_its_group(ctx, bad, n, p, c):
    """Several launches, and one launch of wide vectors."""
    banner(f"group norm with a {bad}, {n} x {p} x {c}")
    x, dy = features(3, n, p, c, torch.float32), normal(4, (n, p, c))
    clean = both(ctx, x, None, None, c // 6, "silu", dy)
    x2 = x.clone()
    x2[1, 350, 13] = bad  # group 2 of image 1
    y, stats, dx, _, _ = both(ctx, x2, None, None, c // 6, "silu", dy)
    hit = torch.zeros(n, c // 6, dtype=torch.bool)
    hit[1, 2] = True
    assert torch.equal(stats[..., 1].isnan().cpu(), hit)
    wide = hit.repeat_interleave(6, 1)[:, None, :].expand(n, p, c)
    for got, ref in ((y, clean[0]), (dx, clean[2])):
        assert got.cpu()[wide].isnan().all() and torch.equal(got.cpu()[~wide], ref.cpu()[~wide])


@pytest.mark.parametrize("n,h,w", [(2, 100, 85), (160, 12, 10)], ids=str)
def test_strided_and_in_place(ctx, bare, n, h, w):
    """Channel slices off 16-byte boundaries, images broadcast, y over x and dx over dy, on several launches and on one of
    wide vectors."""
    from differentiable_gaussian_splatting_amd import gsr
    banner(f"group norm strided, in place, {n} x {h} x {w}")
    wide = features(3, n, h * w, 80, torch.bfloat16).reshape(n, h, w, 80).cuda()
    x = wide[..., 3:51]
    dy = normal(4, (n, h, w, 48), torch.bfloat16).cuda()
    gamma, beta = normal(5, (48,)).cuda(), normal(6, (48,)).cuda()
    xc = x.contiguous()
    assert one_launch(bare, xc, 4) == (n == 160)
    ref = both(ctx, xc.cpu().reshape(n, h * w, 48), gamma.cpu(), beta.cpu(), 4, "silu", dy.cpu().reshape(n, h * w, 48))
    check(ref, xc.cpu().reshape(n, h * w, 48), gamma.cpu(), beta.cpu(), 4, "silu", dy.cpu().reshape(n, h * w, 48))
    y, stats = gsr.gsr_group_norm_forward(ctx, x, gamma, beta, 4, 1e-5, 1)
    assert torch.equal(y.reshape(ref[0].shape), ref[0]) and torch.equal(stats, ref[1])
    dx, dg, db = gsr.gsr_group_norm_backward(ctx, x, gamma, beta, 4, stats, dy, 1)
    assert torch.equal(dx.reshape(ref[2].shape), ref[2]) and torch.equal(dg, ref[3]) and torch.equal(db, ref[4])
    keep = dy.clone()
    gsr.gsr_group_norm_backward(ctx, x, gamma, beta, 4, stats, keep, 1, dx=keep)
    assert torch.equal(keep, dx)
    before = wide.clone()
    gsr.gsr_group_norm_forward(ctx, x, gamma, beta, 4, 1e-5, 1, y=x)
    assert torch.equal(x, y)
    assert torch.equal(wide[..., :3], before[..., :3]) and torch.equal(wide[..., 51:], before[..., 51:])
    b = xc[:1].expand(n, h, w, 48)
    yb, _ = gsr.gsr_group_norm_forward(ctx, b, gamma, beta, 4, 1e-5, 1)
    assert torch.equal(yb, y[:1].expand(n, h, w, 48))


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_the_backward_in_one_launch_asks_for_the_images_sums_alone(ctx, dtype):
    """Two floats per image and channel, and nothing for one image."""
    from differentiable_gaussian_splatting_amd import gsr
    banner(f"group norm backward scratch {dtype}")
    for n, p, c, room in ((1, 40, 24, 1), (160, 120, 48, 8 * 160 * 48)):
        x, dy = features(3, n, p, c, DTYPES[dtype]).cuda(), normal(4, (n, p, c), DTYPES[dtype]).cuda()
        y, st = gsr.gsr_group_norm_forward(ctx, x, None, None, 4, 1e-5, 1)
        ref = gsr.gsr_group_norm_backward(ctx, x, None, None, 4, st, dy, 1)
        tight = gsr.Context(0)
        try:
            gsr.gsr_set_option(tight, gsr.GSR_OPT_ARENA_LIMIT, room)
            got = gsr.gsr_group_norm_backward(tight, x, None, None, 4, st, dy, 1)
            assert all(torch.equal(a, b) for a, b in zip(got, ref))
        finally:
            tight.close()


@pytest.mark.parametrize("n,p", [(2, MANY), (160, 120)], ids=str)
def test_optional_outputs(ctx, n, p):
    """Each output of the backward alone has the values that all three together have."""
    from differentiable_gaussian_splatting_amd import gsr
    banner(f"group norm optional outputs, {n} x {p}")
    x, dy = features(3, n, p, 48, torch.float32).cuda(), normal(4, (n, p, 48)).cuda()
    y, st = gsr.gsr_group_norm_forward(ctx, x, None, None, 4, 1e-5, 1)
    ref = gsr.gsr_group_norm_backward(ctx, x, None, None, 4, st, dy, 1)
    d = gsr._group_norm_desc(ctx, x, None, None, 4, 0.0, 1)
    d.dy_stride[:] = d.dx_stride[:] = d.x_stride[:]
    ptr = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())  # noqa: E731
    for use in ((False, True, False), (False, False, True), (True, False, False), (False, True, True)):
        got = [torch.empty_like(t) if u else None for t, u in zip(ref, use)]
        assert gsr.load().gsr_group_norm_backward(ctx.handle, gsr._stream(None), ctypes.byref(d), ptr(x), None, None,
                                                  ptr(st), ptr(dy), *[ptr(t) for t in got]) == 0
        torch.cuda.synchronize()
        assert all(g is None or torch.equal(g, r) for g, r in zip(got, ref))
