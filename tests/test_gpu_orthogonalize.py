"""GPU orthogonalised updates and the optimiser step on them against the fp64 oracle (oracle/features.py).

Bars. float32 and float16 results: every number is kept to 22 bits where float32 keeps 24, so that each rounding is at
most four times a float32 evaluation's; the error's norm is at most four times that of the same steps in float32 on the
CPU (whose own error is taken as at least one rounding, 2^-24 of the norm, a step: it may be smaller by luck for tiny
matrices), plus the result's own rounding. bfloat16 results: oracle newton_schulz_error's size of the left factors'
roundings (u = 2^-11, A from X's hi), plus the rounding. No element is further off than 12 times the bar's mean size."""
import ctypes
import math

import pytest
import torch

from featurehelp import DTYPES, normal
from gpuhelp import banner
from oracle import features as of

pytestmark = pytest.mark.gpu
QUINTIC = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def ctx():
    from differentiable_gaussian_splatting_amd import gsr
    c = gsr.Context(0)
    yield c
    c.close()


def gradient(seed, batch, m, n, dtype=torch.float32, kind="flat", scale=1e-3):
    if kind == "flat":
        g = normal(seed, (batch, m, n))
    elif kind == "low rank":
        k = min(m, n, 6)
        g = normal(seed, (batch, m, k)) @ normal(seed + 1, (batch, k, n)) + 0.02 * normal(seed + 2, (batch, m, n))
    else:  # steep: singular values fall by 10^-3 over the rank
        u, _, v = torch.linalg.svd(normal(seed, (batch, m, n)), full_matrices=False)
        r = min(m, n)
        g = (u * 10.0 ** (-3 * torch.arange(r) / r)) @ v
    return (scale * g).to(dtype)


def bar(g, steps, dtype, want):
    norm = float(want.norm())
    if dtype == torch.bfloat16:
        e = of.newton_schulz_error(g, steps, 2.0 ** -11, True)
    else:
        plain = float((of.newton_schulz(g, steps, 0.0, torch.float32).double() - want).norm())
        e = 4 * max(plain, len(steps) * 2.0 ** -24 * norm)
    return e


def check(g, got, steps, what, eps=0.0, rounded=True):
    """Each matrix of `got` against the oracle's for g (both [b, m, n])."""
    worst = 0.0
    for gi, oi in zip(g.detach().cpu().double(), got.detach().cpu().double()):
        want = of.newton_schulz(gi, steps, eps)
        norm = float(want.norm())
        e = bar(gi, steps, got.dtype, want) + (of.ROUND[got.dtype] * norm if rounded else 0.0)
        err = oi - want
        worst = max(worst, float(err.norm()) / max(e, 1e-300))
        rms = e / math.sqrt(want.numel())
        assert float(err.abs().max()) <= 12 * rms + of.ROUND[got.dtype] * float(want.abs().max()), what
    print(f"  {what}: worst error / bar {worst:.3g}", flush=True)
    assert worst <= 1.0, (what, worst)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("batch,m,n", [
    (1, 1, 1), (2, 1, 7), (3, 5, 1), (2, 10, 64), (1, 63, 65), (4, 64, 64), (2, 192, 64), (1, 128, 128), (2, 129, 40),
    (1, 96, 513), (2, 200, 333), (1, 700, 130), (1, 512, 512), (1, 520, 640), (2, 513, 1100), (1, 30, 5000),
    (2, 65, 64), (3, 100, 300), (1, 128, 129), (2, 1500, 33), (1, 120, 2050), (1, 4000, 128), (2, 64, 129), (1, 127, 127), (2, 64, 256), (1, 511, 50),
    (3, 17, 300), (1, 64, 513), (2, 9000, 70), (1, 90, 600), (1, 200, 4100), (1, 2500, 300), (1, 513, 2100)])
def test_sizes(ctx, dtype, batch, m, n):
    from differentiable_gaussian_splatting_amd import gsr
    banner(f"orthogonalize {dtype} {batch} x {m} x {n}")
    g = gradient(m + n, batch, m, n, DTYPES[dtype])
    out = gsr.gsr_orthogonalize(ctx, g.cuda(), eps=0.0)
    assert out.dtype == g.dtype and out.shape == g.shape
    check(g, out, [QUINTIC] * 5, f"{dtype} {batch}x{m}x{n}")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("kind", ["low rank", "steep"])
@pytest.mark.parametrize("m,n", [(64, 100), (300, 180), (530, 600), (300, 4100)])
def test_decaying_spectra(ctx, dtype, kind, m, n):
    from differentiable_gaussian_splatting_amd import gsr
    banner(f"orthogonalize {dtype} {kind} {m} x {n}")
    g = gradient(1, 2, m, n, DTYPES[dtype], kind)
    check(g, gsr.gsr_orthogonalize(ctx, g.cuda(), eps=0.0), [QUINTIC] * 5, f"{dtype} {kind}")


@pytest.mark.parametrize("m", [48, 200, 600])
@pytest.mark.parametrize("steps", [
    [QUINTIC], [QUINTIC] * 3, [(1.5, -0.5, 0.0)] * 8, [(2.0, -1.5, 0.5)] * 6, [QUINTIC] * 5 + [(1.5, -0.5, 0.0)] * 3,
    [(7.0, 0.0, 0.0), (0.1, -0.001, 0.0)], [(0.0, 0.0, 0.0), QUINTIC]], ids=lambda s: f"{len(s)}x{s[0][0]}")
def test_steps_and_coefficients(ctx, m, steps):
    from differentiable_gaussian_splatting_amd import gsr
    banner(f"orthogonalize of {len(steps)} steps from {steps[0]}, {m}")
    g = gradient(5, 2, m, m + 30)
    check(g, gsr.gsr_orthogonalize(ctx, g.cuda(), len(steps), steps, 0.0), steps, f"{steps[0]}")


@pytest.mark.parametrize("m", [40, 300])
def test_singular_values(ctx, m):
    """What it is for: the result's singular values near 1, its singular vectors those of the gradient."""
    from differentiable_gaussian_splatting_amd import gsr
    banner(f"orthogonalize: singular values, {m}")
    g = gradient(9, 1, m, 2 * m)
    out = gsr.gsr_orthogonalize(ctx, g.cuda())[0].cpu().double()
    want = of.newton_schulz_svd(g[0], [QUINTIC] * 5, 1e-7)
    assert float((out - want).norm() / want.norm()) < 1e-4
    s = torch.linalg.svdvals(out)
    assert 0.6 < float(s.min()) and float(s.max()) < 1.25


@pytest.mark.parametrize("m,n", [(40, 72), (300, 180)])
def test_scales_zeros_and_bad_values(ctx, m, n):
    from differentiable_gaussian_splatting_amd import gsr
    banner(f"orthogonalize of zeros, infinities, tiny and huge matrices, {m} x {n}")
    steps = [QUINTIC] * 5
    for scale in (1e-30, 1e-10, 1e25, 1e36):
        g = gradient(3, 1, m, n, scale=scale)
        check(g, gsr.gsr_orthogonalize(ctx, g.cuda(), eps=0.0), steps, f"scale {scale}")
    g = gradient(3, 1, m, n, scale=1e-8)
    check(g, gsr.gsr_orthogonalize(ctx, g.cuda(), eps=1e-6), steps, "eps as large as the norm", 1e-6)
    g = gradient(4, 5, m, n)
    clean = gsr.gsr_orthogonalize(ctx, g.cuda())
    g[0] = 0
    g[2, m // 2, n // 3] = float("nan")
    g[3, 0, 0] = float("inf")
    for eps in (0.0, 1e-7):
        out = gsr.gsr_orthogonalize(ctx, g.cuda(), eps=eps)
        assert (out[0] == 0).all() and out[2].isnan().all() and out[3].isnan().all()
        if eps:
            assert torch.equal(out[1], clean[1]) and torch.equal(out[4], clean[4])


# tiles of 64 to 256, in both kinds of products, by the number of matrices; odd counts of tiles; two steps at a time
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,m,n", [
    (16, 520, 640), (40, 520, 640), (64, 500, 500), (85, 500, 500), (24, 1900, 600), (3, 1100, 1030), (7, 300, 2500)])
def test_stacks(ctx, dtype, batch, m, n):
    """Copies of three matrices: the copies have the same bits, the three are held to the oracle. (Bits differ between
    stacks of other sizes: a tile on the diagonal adds hi lo before lo hi on both of its sides, mirrored tiles on one.)"""
    from differentiable_gaussian_splatting_amd import gsr
    banner(f"orthogonalize {dtype} {batch} x {m} x {n}, copies")
    few = gradient(2, 3, m, n, DTYPES[dtype]).cuda()
    stack = few.repeat(batch // 3 + 1, 1, 1)[:batch]
    for steps in (2, 5):
        got = gsr.gsr_orthogonalize(ctx, stack, steps)
        for i in range(batch):
            assert torch.equal(got[i], got[i % 3]), i
        check(few, got[:3], [QUINTIC] * steps, f"{dtype} of {batch}, {steps} steps", 1e-7)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,n", [(40, 72), (72, 40), (300, 180), (530, 650), (70, 900), (260, 1200)])
def test_strided_broadcast_in_place_repeated(ctx, dtype, m, n):
    from differentiable_gaussian_splatting_amd import gsr
    banner(f"orthogonalize strided, in place, repeated, {dtype} {m} x {n}")
    wide = gradient(1, 3, m + 2, n + 11, DTYPES[dtype]).cuda()
    g = wide[:, 1:-1, 5:n + 5]
    ref = gsr.gsr_orthogonalize(ctx, g.contiguous())
    assert torch.equal(gsr.gsr_orthogonalize(ctx, g), ref)
    assert torch.equal(gsr.gsr_orthogonalize(ctx, g[1]), ref[1])
    turned = torch.empty((m, 3, n), dtype=g.dtype, device="cuda").transpose(0, 1)  # rows further apart than matrices
    assert torch.equal(gsr.gsr_orthogonalize(ctx, g, out=turned), ref)
    same = gsr.gsr_orthogonalize(ctx, g[:1].expand(4, m, n))
    assert all(torch.equal(same[i], ref[0]) for i in range(4))
    before = wide.clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        again = gsr.gsr_orthogonalize(ctx, g, stream=s)
        s.synchronize()
        assert torch.equal(again, ref)
    assert torch.equal(wide, before)
    gsr.gsr_orthogonalize(ctx, g, out=g)
    assert torch.equal(g, ref)
    wide[:, 1:-1, 5:n + 5] = before[:, 1:-1, 5:n + 5]
    assert torch.equal(wide, before)


@pytest.mark.parametrize("m,n", [(40, 72), (300, 180), (70, 900), (1200, 260)])
def test_graph_replays(ctx, m, n):
    from differentiable_gaussian_splatting_amd import gsr
    banner(f"orthogonalize and step in a graph, {m} x {n}")
    g, p0 = gradient(1, 2, m, n).cuda(), normal(2, (2, m, n)).cuda()
    ref = gsr.gsr_orthogonalize(ctx, g)
    want_p, want_m = p0.clone(), torch.zeros_like(p0)
    for _ in range(3):
        gsr.gsr_muon_step(ctx, want_p, g, want_m, 0.02)
    out, p, mom = torch.empty_like(g), p0.clone(), torch.zeros_like(p0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gsr.gsr_orthogonalize(ctx, g, out=out)
        gsr.gsr_muon_step(ctx, p, g, mom, 0.02)
    for _ in range(3):
        out.fill_(7.0)
        gsr.gsr_orthogonalize(ctx, g[:1, :20])  # the same arena, other contents
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
    assert torch.equal(p, want_p) and torch.equal(mom, want_m)


@pytest.mark.parametrize("grad", list(DTYPES))
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("batch,m,n", [(2, 64, 64), (1, 192, 64), (3, 10, 64), (2, 150, 333), (1, 640, 520), (2, 100, 700),
                                       (1, 1100, 90), (60, 256, 140)])
def test_muon_step(ctx, grad, nesterov, batch, m, n):
    from differentiable_gaussian_splatting_amd import gsr
    banner(f"muon step {grad} nesterov {nesterov} {batch} x {m} x {n}")
    lr, mu, decay = 0.03, 0.9, 0.99
    steps = [QUINTIC] * 5
    p = normal(1, (batch, m, n)).cuda()
    mom = gradient(2, batch, m, n, scale=5e-3).cuda()
    for turn in range(2):  # the second step on the first one's state
        g = gradient(3 + turn, batch, m, n, DTYPES[grad])
        p0, m0 = p.cpu().double(), mom.cpu().double()
        gsr.gsr_muon_step(ctx, p, g.cuda(), mom, lr, mu, nesterov, decay, eps=0.0)
        m1 = mu * m0 + g.double()
        # two roundings: mu in float32, the fused product and sum
        assert ((mom.cpu().double() - m1).abs() <= of.U32 * (2 * (mu * m0).abs() + m1.abs())).all()
        m1 = mom.cpu().double()
        u = (g.double() + mu * m1 if nesterov else m1).float()
        for i in range(batch):
            want = of.newton_schulz(u[i].double(), steps)
            e = bar(u[i], steps, torch.float32, want)
            whole = decay * p0[i] - lr * want
            # u's own roundings (one, and mu's) reach the result like those of a float32 evaluation's first step
            off = p[i].cpu().double() - whole
            rounding = 3 * of.U32 * float(p0[i].norm() + lr * want.norm())
            assert float(off.norm()) <= lr * 1.5 * e + rounding, (turn, i)
            assert float(off.abs().max()) <= 12 * lr * 1.5 * e / math.sqrt(m * n) + \
                3 * of.U32 * float(p0[i].abs().max() + lr), (turn, i)


def test_muon_step_of_strided_stacks(ctx):
    from differentiable_gaussian_splatting_amd import gsr
    banner("muon step of strided parameters")
    for m, n in ((40, 72), (300, 180), (70, 900), (900, 70)):
        big_p, big_m = normal(1, (3, m + 3, n + 5)).cuda(), normal(2, (3, m + 1, n + 2)).cuda()
        big_g = gradient(3, 3, m, n + 9, torch.bfloat16).cuda()
        p, mom, g = big_p[:, 2:-1, 3:n + 3], big_m[:, 1:, 1:n + 1], big_g[:, :, 4:n + 4]
        pc, mc = p.clone(), mom.clone()
        keep_p, keep_m, keep_g = big_p.clone(), big_m.clone(), big_g.clone()
        gsr.gsr_muon_step(ctx, pc, g.contiguous(), mc, 0.1, decay=0.9)
        gsr.gsr_muon_step(ctx, p, g, mom, 0.1, decay=0.9)
        assert torch.equal(p, pc) and torch.equal(mom, mc) and torch.equal(big_g, keep_g)
        keep_p[:, 2:-1, 3:n + 3], keep_m[:, 1:, 1:n + 1] = pc, mc  # nothing else was written
        assert torch.equal(big_p, keep_p) and torch.equal(big_m, keep_m)
        one_p, one_m = keep_p[1, 2:-1, 3:n + 3].clone(), keep_m[1, 1:, 1:n + 1].clone()
        gsr.gsr_muon_step(ctx, one_p, g[1], one_m, 0.1)
        gsr.gsr_muon_step(ctx, p[1:2], g[1:2], mom[1:2], 0.1)
        assert torch.equal(one_p, p[1]) and torch.equal(one_m, mom[1])


def test_zero_gradients_move_nothing_but_the_decay(ctx):
    from differentiable_gaussian_splatting_amd import gsr
    banner("muon step of zero gradients")
    p, m = normal(1, (2, 30, 50)).cuda(), torch.zeros((2, 30, 50), device="cuda")
    want = 0.5 * p
    gsr.gsr_muon_step(ctx, p, torch.zeros_like(p), m, 0.1, decay=0.5)
    assert torch.equal(p, want) and (m == 0).all()


def test_empty_and_kernel_times(ctx):
    from differentiable_gaussian_splatting_amd import gsr
    banner("orthogonalize of nothing; kernel times")
    for shape in ((0, 4, 5), (2, 0, 5), (2, 4, 0)):
        g = torch.empty(shape, device="cuda")
        assert gsr.gsr_orthogonalize(ctx, g).shape == g.shape
        gsr.gsr_muon_step(ctx, g, g.clone(), g.clone(), 0.1)
    c = gsr.Context(0)
    try:
        gsr.gsr_set_option(c, gsr.GSR_OPT_KERNEL_TIMING, 4)
        g = gradient(1, 1, 90, 200).cuda()
        gsr.gsr_orthogonalize(c, g)
        gsr.gsr_muon_step(c, g.clone(), g, torch.zeros_like(g), 0.1)
        for stage in (gsr.GSR_STAGE_ORTHOGONALIZE, gsr.GSR_STAGE_MUON):
            t = gsr.gsr_kernel_times(c, stage)
            assert len(t) == 1 and 0 < t[0] < 1000
    finally:
        c.close()


def test_refusals(ctx):
    from differentiable_gaussian_splatting_amd import gsr
    banner("orthogonalize refusals")
    g = torch.ones((2, 10, 12), device="cuda")
    orth = lambda *a, **k: gsr.gsr_orthogonalize(ctx, *a, **k)  # noqa: E731
    for kw in ({"eps": -1.0}, {"eps": float("nan")}, {"coefficients": (float("inf"), 0, 0)}, {"coefficients": (9, 0, 0)},
               {"coefficients": (3.0, 0, 0)}, {"coefficients": (0.0, 0.0, 8.1)}):
        with pytest.raises(gsr.GsrError) as e:
            orth(g, **kw)
        assert e.value.status == gsr.GSR_EINVAL
    for kw in ({"steps": 0}, {"steps": 9}, {"coefficients": (1, 2)}, {"coefficients": [QUINTIC] * 4}):
        with pytest.raises(ValueError):
            orth(g, **kw)
    with pytest.raises(gsr.GsrError, match="overlap"):
        orth(g, out=torch.zeros((1, 10, 12), device="cuda").expand(2, 10, 12))
    with pytest.raises(TypeError):
        orth(g.double())
    with pytest.raises(TypeError):
        orth(g, out=g.half())
    for bad in (g.cpu(), g[0, 0], g.transpose(1, 2), g[None]):
        with pytest.raises(ValueError):
            orth(bad)
    with pytest.raises(ValueError):
        orth(g, out=g[:1])
    p, m = g.clone(), g.clone()
    muon = lambda *a, **k: gsr.gsr_muon_step(ctx, *a, **k)  # noqa: E731
    for kw in ({"lr": float("nan")}, {"lr": 0.1, "mu": float("inf")}, {"lr": 0.1, "decay": float("nan")}):
        with pytest.raises(gsr.GsrError) as e:
            muon(p, g, m, **kw)
        assert e.value.status == gsr.GSR_EINVAL
    with pytest.raises(TypeError):
        muon(p.half(), g, m, 0.1)
    with pytest.raises(TypeError):
        muon(p, g, m.half(), 0.1)
    with pytest.raises(ValueError):
        muon(p[:1], g, m, 0.1)
    for args in ((g[:1].expand(2, 10, 12), g, m), (p, g, g[:1].expand(2, 10, 12))):
        with pytest.raises(gsr.GsrError, match="overlap"):
            muon(*args, 0.1)
    assert torch.equal(p, g) and torch.equal(m, g)
    lib, h = gsr.load(), ctx.handle

    def desc(dtype=0, batch=1, rows=4, cols=4, steps=5):
        d = gsr.gsr_newton_schulz(dtype, batch, rows, cols, steps, 1e-7)
        for k in range(8):
            d.coefficients[k][:] = QUINTIC
        return d
    at = ctypes.c_void_p(g.data_ptr())
    for d, want in ((desc(3), gsr.GSR_EINVAL), (desc(steps=0), gsr.GSR_EINVAL), (desc(steps=9), gsr.GSR_EINVAL),
                    (desc(batch=1 << 16), gsr.GSR_EOVERFLOW), (desc(rows=1 << 20), gsr.GSR_EOVERFLOW),
                    (desc(rows=1 << 16, cols=1 << 15), gsr.GSR_EOVERFLOW), (desc(batch=2), gsr.GSR_EINVAL)):
        assert lib.gsr_orthogonalize(h, None, ctypes.byref(d), at, at) == want
        assert lib.gsr_muon_step(h, None, ctypes.byref(d), at, at, at, 0.1, 0.9, 1, 1.0) == want
    assert lib.gsr_orthogonalize(h, None, None, at, at) == gsr.GSR_EINVAL
    assert lib.gsr_orthogonalize(h, None, ctypes.byref(desc()), None, at) == gsr.GSR_EINVAL
    assert lib.gsr_orthogonalize(h, None, ctypes.byref(desc()), at, ctypes.c_void_p(g.data_ptr() + 2)) == gsr.GSR_EINVAL
    assert lib.gsr_muon_step(h, None, ctypes.byref(desc()), at, None, at, 0.1, 0.9, 1, 1.0) == gsr.GSR_EINVAL


def test_the_arena_limit_refuses_and_leaves_the_state(ctx):
    from differentiable_gaussian_splatting_amd import gsr
    banner("muon step beyond the arena limit")
    c = gsr.Context(0)
    try:
        gsr.gsr_set_option(c, gsr.GSR_OPT_ARENA_LIMIT, 1 << 16)
        g, p, m = gradient(1, 1, 300, 300).cuda(), normal(2, (1, 300, 300)).cuda(), torch.zeros((1, 300, 300)).cuda()
        keep = p.clone()
        with pytest.raises(gsr.GsrError) as e:
            gsr.gsr_muon_step(c, p, g, m, 0.1)
        assert e.value.status == gsr.GSR_ENOMEM
        assert torch.equal(p, keep) and (m == 0).all()
    finally:
        c.close()


def test_no_coefficients_are_refused(ctx):
    from differentiable_gaussian_splatting_amd import gsr
    g = torch.ones(4, 4, device="cuda")
    for table in ((), [(1.0, 0.0)] * 5, [(1.0, 0.0, 0.0)] * 4):
        with pytest.raises(ValueError, match="coefficients"):
            gsr.gsr_orthogonalize(ctx, g, 5, table)
