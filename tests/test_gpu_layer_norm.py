"""GPU layer norm against the fp64 oracle (oracle/features.py), element by element within the oracle's float32 error
bound plus the result's own rounding to its type."""
import ctypes

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


def tokens(seed, rows, c, dtype, centre=0.7):
    """Each channel with a centre and a scale of its own, each token with a length of its own."""
    x = normal(seed, (rows, c)) * (0.5 + normal(seed + 1, (c,)).abs()) + centre * normal(seed + 2, (c,))
    return (x * torch.exp(0.5 * normal(seed + 3, (rows, 1)))).to(dtype)


def check(x, gamma, beta, dy, got, eps=1e-5):
    x, dy = x.reshape(-1, x.shape[-1]), dy.reshape(-1, x.shape[-1])
    r = of.layer_norm(x.double(), None if gamma is None else gamma.double(), None if beta is None else beta.double(), eps,
                      dy.double())
    u, tiny = of.ROUND[x.dtype], of.TINY[x.dtype]
    y, stats, dx, dgamma, dbeta = got
    stats = stats.reshape(-1, 2)
    within(stats[:, 0], r["mean"], r["e_mean"], "mean")
    within(stats[:, 1], r["rstd"], r["e_rstd"], "rstd")
    for name, t in (("y", y), ("dx", dx)):
        within(t.reshape(x.shape), r[name], r["e_" + name] + u * r[name].abs() + tiny, name)
    within(dgamma, r["dgamma"], r["e_dgamma"] + of.U32 * r["dgamma"].abs(), "dgamma")
    within(dbeta, r["dbeta"], r["e_dbeta"] + of.U32 * r["dbeta"].abs(), "dbeta")


def both(ctx, x, gamma, beta, dy, eps=1e-5, **kw):
    from differentiable_gaussian_splatting_amd import gsr
    d = lambda t: None if t is None else t.cuda()  # noqa: E731
    y, stats = gsr.gsr_layer_norm_forward(ctx, d(x), d(gamma), d(beta), eps, **kw)
    return (y, stats) + gsr.gsr_layer_norm_backward(ctx, d(x), d(gamma), stats, d(dy), **kw)


# every team and number of vectors of either element size, their edges, and the form that reads tokens again
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,c", [
    (1, 1), (3, 2), (5, 7), (969, 90), (64, 32), (65, 33), (7, 64), (300, 65), (17, 128), (9, 129), (130, 256), (33, 257),
    (2500, 512), (70, 513), (1, 1024), (40, 1024), (11, 1025), (600, 640), (5, 1536), (3, 1537), (6, 2048), (4, 2052),
    (5, 4096), (2, 4099), (3, 8192), (2, 8193), (2, 16384), (3, 16385), (70, 20001), (1, 50000), (20000, 8)])
def test_sizes(ctx, dtype, rows, c):
    banner(f"layer norm {dtype} {rows}x{c}")
    t = DTYPES[dtype]
    x, dy = tokens(rows + c, rows, c, t), normal(rows, (rows, c), t)
    gamma, beta = 1 + 0.2 * normal(1, (c,)), normal(2, (c,))
    check(x, gamma, beta, dy, both(ctx, x, gamma, beta, dy))


@pytest.mark.parametrize("c", [24, 640, 3000, 20000])
def test_without_affine(ctx, c):
    banner(f"layer norm without gamma and beta, {c}")
    x, dy = tokens(3, 50, c, torch.float32), normal(4, (50, c))
    check(x, None, None, dy, both(ctx, x, None, None, dy))


@pytest.mark.parametrize("c", [24, 640, 3000, 20000])
def test_a_far_mean_and_an_outlier_cost_no_variance(ctx, c):
    banner(f"layer norm of a far mean, of an outlier, {c}")
    x = 1000 + normal(1, (20, c))
    x[:10, 0] = 1e5
    check(x, None, None, normal(2, (20, c)), both(ctx, x, None, None, normal(2, (20, c))))


def test_constant_tokens(ctx):
    from differentiable_gaussian_splatting_amd import gsr
    banner("layer norm of constants")
    for c in (12, 500, 5000, 20000):
        y, stats = gsr.gsr_layer_norm_forward(ctx, torch.full((7, c), 3.25, device="cuda"))
        assert (y == 0).all() and (stats[:, 0] == 3.25).all()
        assert torch.allclose(stats[:, 1].cpu(), torch.tensor(1e-5).rsqrt(), rtol=1e-6)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("c", [24, 700, 2500, 20000])
def test_a_bad_value_stays_in_its_token(ctx, bad, c):
    banner(f"layer norm with a {bad}, {c}")
    x, dy = tokens(3, 37, c, torch.float32), normal(4, (37, c))
    clean = both(ctx, x, None, None, dy)
    x2 = x.clone()
    x2[11, c // 2] = bad
    y, stats, dx, dgamma, dbeta = both(ctx, x2, None, None, dy)
    hit = torch.zeros(37, dtype=torch.bool)
    hit[11] = True
    assert torch.equal(stats[:, 1].isnan().cpu(), hit)
    for got, ref in ((y, clean[0]), (dx, clean[2])):
        assert got.cpu()[hit].isnan().all() and torch.equal(got.cpu()[~hit], ref.cpu()[~hit])
    assert dgamma.isnan().all() and torch.equal(dbeta, clean[4])


@pytest.mark.parametrize("c", [24, 600, 2500, 20000])
def test_strided_broadcast_and_in_place(ctx, c):
    from differentiable_gaussian_splatting_amd import gsr
    banner(f"layer norm strided, broadcast, in place, {c}")
    wide = tokens(3, 6 * 11, c + 16, torch.bfloat16).reshape(6, 11, c + 16).cuda()
    x = wide[..., 3:c + 3]  # a channel slice, not 16-byte aligned
    dy = normal(4, (6, 11, c), torch.bfloat16).cuda()
    gamma, beta = normal(5, (c,)).cuda(), normal(6, (c,)).cuda()
    y, stats = gsr.gsr_layer_norm_forward(ctx, x, gamma, beta)
    assert stats.shape == (6, 11, 2)
    xc = x.contiguous()
    y2, stats2 = gsr.gsr_layer_norm_forward(ctx, xc, gamma, beta)
    assert torch.equal(y, y2) and torch.equal(stats, stats2)
    ref = gsr.gsr_layer_norm_backward(ctx, xc, gamma, stats, dy)
    flipped = dy.transpose(0, 1).contiguous().transpose(0, 1)  # tokens further apart than batch entries
    got = gsr.gsr_layer_norm_backward(ctx, x, gamma, stats, flipped)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    keep = dy.clone()
    gsr.gsr_layer_norm_backward(ctx, x, gamma, stats, keep, dx=keep)
    assert torch.equal(keep, ref[0])
    before = wide.clone()
    gsr.gsr_layer_norm_forward(ctx, x, gamma, beta, y=x)
    assert torch.equal(x, y)
    assert torch.equal(wide[..., :3], before[..., :3]) and torch.equal(wide[..., c + 3:], before[..., c + 3:])
    b = xc[:1].expand(3, 11, c)
    yb, _ = gsr.gsr_layer_norm_forward(ctx, b, gamma, beta)
    assert all(torch.equal(yb[i], y[0]) for i in range(3))
    # one token, two leading dimensions more
    one, _ = gsr.gsr_layer_norm_forward(ctx, xc[2, 3].reshape(1, 1, 1, c), gamma, beta)
    assert torch.equal(one.reshape(c), y[2, 3])


@pytest.mark.parametrize("rows,c", [(5000, 48), (33, 1000), (300, 4000), (3, 20000)], ids=str)
def test_repeats_on_another_stream(ctx, rows, c):
    from differentiable_gaussian_splatting_amd import gsr
    banner(f"layer norm on another stream, repeated, {rows} x {c}")
    x, dy = tokens(3, rows, c, torch.float16).cuda(), normal(4, (rows, c), torch.float16).cuda()
    y, st = gsr.gsr_layer_norm_forward(ctx, x)
    ref = gsr.gsr_layer_norm_backward(ctx, x, None, st, dy)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        y2, st2 = gsr.gsr_layer_norm_forward(ctx, x, stream=s)
        got = gsr.gsr_layer_norm_backward(ctx, x, None, st2, dy, stream=s)
        s.synchronize()
        assert torch.equal(y, y2) and torch.equal(st, st2) and all(torch.equal(a, b) for a, b in zip(ref, got))


@pytest.mark.parametrize("rows,c", [(3000, 48), (33, 1000), (3, 20000)], ids=str)
def test_graph_replays(ctx, rows, c):
    from differentiable_gaussian_splatting_amd import gsr
    banner(f"layer norm in a graph, {rows} x {c}")
    x, dy = tokens(3, rows, c, torch.float32).cuda(), normal(4, (rows, c)).cuda()
    gamma, beta = normal(5, (c,)).cuda(), normal(6, (c,)).cuda()
    y, st = gsr.gsr_layer_norm_forward(ctx, x, gamma, beta)
    ref = [t.clone() for t in (y, st) + gsr.gsr_layer_norm_backward(ctx, x, gamma, st, dy)]
    bufs = [torch.empty_like(t) for t in ref]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gsr.gsr_layer_norm_forward(ctx, x, gamma, beta, y=bufs[0], stats=bufs[1])
        gsr.gsr_layer_norm_backward(ctx, x, gamma, bufs[1], dy, *bufs[2:])
    for i in range(3):
        for b in bufs:
            b.fill_(float(i))
        both(ctx, x.cpu()[:2], None, None, dy.cpu()[:2])  # the same arena, other contents
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, bufs)), i


def test_no_tokens_and_optional_outputs(ctx):
    from differentiable_gaussian_splatting_amd import gsr
    banner("layer norm of nothing")
    for shape in ((0, 5, 12), (3, 0, 12)):
        x = torch.empty(shape, device="cuda")
        y, st = gsr.gsr_layer_norm_forward(ctx, x)
        assert y.shape == x.shape
        out = gsr.gsr_layer_norm_backward(ctx, x, None, st, x, dgamma=torch.ones(12, device="cuda"),
                                          dbeta=torch.ones(12, device="cuda"))
        assert (out[1] == 0).all() and (out[2] == 0).all()
    x = torch.empty((3, 4, 0), device="cuda")
    assert gsr.gsr_layer_norm_forward(ctx, x)[0].shape == x.shape
    p = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())  # noqa: E731
    for c in (24, 1500, 20000):  # each output alone gives the same values
        x, dy = tokens(3, 300, c, torch.float32).cuda(), normal(4, (300, c)).cuda()
        y, st = gsr.gsr_layer_norm_forward(ctx, x)
        ref = gsr.gsr_layer_norm_backward(ctx, x, None, st, dy)
        d = gsr._layer_norm_desc(ctx, x, None, None, 0.0)
        d.dy_stride[:] = d.dx_stride[:] = d.x_stride[:]
        for use in ((False, True, False), (False, False, True), (True, False, False), (False, False, False)):
            got = [torch.empty_like(t) if u else None for t, u in zip(ref, use)]
            assert gsr.load().gsr_layer_norm_backward(ctx.handle, gsr._stream(None), ctypes.byref(d), p(x), None, p(st),
                                                      p(dy), *[p(t) for t in got]) == 0
            torch.cuda.synchronize()
            assert all(g is None or torch.equal(g, r) for g, r in zip(got, ref)), (c, use)


def test_offsets_past_32_bits(ctx):
    """More than 2^32 elements: the last tokens are their own, forward and backward."""
    from differentiable_gaussian_splatting_amd import gsr
    banner("layer norm of (2^21 + 5) x 2056 (26 GB)")
    rows, c = (1 << 21) + 5, 2056
    few = tokens(1, 64, c, torch.bfloat16).cuda()
    x = few.repeat(rows // 64 + 1, 1)[:rows]
    y, st = gsr.gsr_layer_norm_forward(ctx, x)
    dx, dgamma, _ = gsr.gsr_layer_norm_backward(ctx, x, None, st, x)
    ref, ref_st = gsr.gsr_layer_norm_forward(ctx, few)
    ref_dx = gsr.gsr_layer_norm_backward(ctx, few, None, ref_st, few)[0]
    for got, want in ((y, ref), (dx, ref_dx), (st, ref_st)):
        whole = got[:rows // 64 * 64].view(-1, 64, got.shape[-1])
        assert torch.equal(whole[-1], want) and torch.equal(whole[whole.shape[0] // 2], want)
        assert torch.equal(got[rows // 64 * 64:], want[:rows % 64])
    del x, y, dx
    torch.cuda.empty_cache()


def test_kernel_times(ctx):
    from differentiable_gaussian_splatting_amd import gsr
    banner("kernel times of layer norm")
    c = gsr.Context(0)
    try:
        gsr.gsr_set_option(c, gsr.GSR_OPT_KERNEL_TIMING, 4)
        x = tokens(1, 100, 64, torch.float32)
        both(c, x, None, None, x)
        for stage in (gsr.GSR_STAGE_LAYER_NORM_FORWARD, gsr.GSR_STAGE_LAYER_NORM_BACKWARD):
            t = gsr.gsr_kernel_times(c, stage)
            assert len(t) == 1 and 0 < t[0] < 1000
    finally:
        c.close()


def test_refusals(ctx):
    from differentiable_gaussian_splatting_amd import gsr
    banner("layer norm refusals")
    x = torch.zeros((2, 10, 12), device="cuda")
    fwd = lambda *a, **k: gsr.gsr_layer_norm_forward(ctx, *a, **k)  # noqa: E731
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(gsr.GsrError) as e:
            fwd(x, None, None, eps)
        assert e.value.status == gsr.GSR_EINVAL
    with pytest.raises(gsr.GsrError, match="overlap"):
        fwd(x, y=torch.zeros((1, 10, 12), device="cuda").expand(2, 10, 12))
    with pytest.raises(TypeError):
        fwd(x.double())
    with pytest.raises(TypeError):
        fwd(x, torch.ones(12, device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError):
        fwd(x, None, torch.ones(11, device="cuda"))
    with pytest.raises(ValueError):
        fwd(x.cpu())
    with pytest.raises(ValueError):
        fwd(x[0, 0])
    with pytest.raises(ValueError, match="adjacent"):
        fwd(x.transpose(1, 2))
    with pytest.raises(ValueError, match="evenly"):
        fwd(torch.zeros((2, 6, 8, 12), device="cuda")[:, :, :5])
    stats = fwd(x)[1]
    back = lambda *a, **k: gsr.gsr_layer_norm_backward(ctx, *a, **k)  # noqa: E731
    with pytest.raises(ValueError):
        back(x, None, stats[:1], x)
    with pytest.raises(ValueError):
        back(x, None, stats, x[:, :5])
    with pytest.raises(TypeError):
        back(x, None, stats, x.half())
    with pytest.raises(gsr.GsrError, match="overlap"):
        back(x, None, stats, x, dx=torch.zeros((1, 10, 12), device="cuda").expand(2, 10, 12))
    n = 1 << 32
    with pytest.raises(gsr.GsrError) as e:
        fwd(x[:1, :1].expand(1, n, 12), y=x, stats=stats)
    assert e.value.status == gsr.GSR_EOVERFLOW
    lib, h = gsr.load(), ctx.handle
    for d, want in ((gsr.gsr_layer_norm(0, 1 << 16, 1 << 15, 4, 1e-5), gsr.GSR_EOVERFLOW),
                    (gsr.gsr_layer_norm(0, 1, 1, 1 << 20, 1e-5), gsr.GSR_EOVERFLOW),
                    (gsr.gsr_layer_norm(3, 1, 1, 4, 1e-5), gsr.GSR_EINVAL),
                    (gsr.gsr_layer_norm(0, 1, 1, 4, 1e-5), gsr.GSR_EINVAL)):
        assert lib.gsr_layer_norm_forward(h, None, ctypes.byref(d), *[None] * 5) == want
        assert lib.gsr_layer_norm_backward(h, None, ctypes.byref(d), None, None, None, None, ctypes.c_void_p(16), None,
                                           None) == want
    assert lib.gsr_layer_norm_forward(h, None, None, *[None] * 5) == gsr.GSR_EINVAL
    d = gsr.gsr_layer_norm(0, 1, 1, 4, 1e-5)
    p = x.data_ptr()
    assert lib.gsr_layer_norm_forward(h, None, ctypes.byref(d), ctypes.c_void_p(p + 2), None, None, ctypes.c_void_p(p),
                                      ctypes.c_void_p(p)) == gsr.GSR_EINVAL
