"""GPU cross attention of visible infinities and NaN under masks: they reach what the formulas say they reach, and
nothing else. The formulas are evaluated in float64 over each query's visible keys alone, so that what is hidden never
enters a sum; which elements are not finite follows from them, the finite ones are held to the oracle's bounds."""
import math

import pytest
import torch

from featurehelp import DTYPES, normal
from gpuhelp import banner
from oracle import features as of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    from differentiable_gaussian_splatting_amd import gsr
    c = gsr.Context(0)
    yield c
    c.close()


def inputs(seed, b, tq, tk, h, hk, d, dtype):
    return (normal(seed, (b, tq, h, d), dtype), normal(seed + 1, (b, tk, hk, d), dtype),
            normal(seed + 2, (b, tk, hk, d), dtype), normal(seed + 3, (b, tq, h, d), dtype))


def formulas(q, k, v, do, mask):
    """o, lse, dq, dk, dv in float64, row by row over the visible keys."""
    q, k, v, do = (t.double() for t in (q, k, v, do))
    B, Tq, H, D = q.shape
    Tk, Hk = k.shape[1], k.shape[2]
    mask = mask.expand(B, H, Tq, Tk)
    o, lse = torch.zeros_like(q), torch.full((B, H, Tq), -math.inf, dtype=torch.float64)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for b in range(B):
        for h in range(H):
            j = h * Hk // H
            for t in range(Tq):
                see = mask[b, h, t].nonzero().flatten()
                if not len(see):
                    continue
                qt, kt, vt, dt = q[b, t, h], k[b, see, j], v[b, see, j], do[b, t, h]
                s = (kt @ qt) * D ** -0.5
                lse[b, h, t] = torch.logsumexp(s, 0)
                p = torch.exp(s - lse[b, h, t])
                o[b, t, h] = (p[:, None] * vt).sum(0)
                ds = D ** -0.5 * p * (vt @ dt - (dt * o[b, t, h]).sum())
                dq[b, t, h] = (ds[:, None] * kt).sum(0)
                dk[b, see, j] += ds[:, None] * qt
                dv[b, see, j] += p[:, None] * dt
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def run(ctx, q, k, v, do, mask):
    from differentiable_gaussian_splatting_amd import gsr
    q, k, v, do = (t.cuda() for t in (q, k, v, do))
    mask = None if mask is None else mask.cuda()
    o, lse = gsr.gsr_cross_attention_forward(ctx, q, k, v, None, None, mask)
    dq, dk, dv = gsr.gsr_cross_attention_backward(ctx, q, k, v, o, lse, do, None, None, mask)
    return dict(zip(("o", "lse", "dq", "dk", "dv"), (t.cpu().double() for t in (o, lse, dq, dk, dv))))


def check(got, want, clean):
    """o and dv have the formulas' infinities and NaN; the gradients through the softmax are finite where theirs are
    (whether a sum of theirs is an infinity or a NaN depends on its order). Finite values within the bounds of the
    problem with the bad elements replaced by zeros, whose finite results are the same."""
    for name in ("o", "dv", "lse", "dq", "dk"):
        g, w = got[name], want[name]
        assert torch.equal(g.isfinite(), w.isfinite()), name
        if name in ("o", "dv"):
            assert torch.equal(g.isnan(), w.isnan()), name
            assert torch.equal(g[g.isinf()], w[w.isinf()]), name
        fine = w.isfinite()
        err, bound = (g - w).abs()[fine], clean["e_" + name].expand(w.shape)[fine]
        worst = float((err / bound.clamp_min(1e-300)).max()) if err.numel() else 0.0
        print(f"  {name}: {int((~fine).sum())} not finite, worst error / bound {worst:.3g}", flush=True)
        assert worst <= 1.0, (name, worst)


def zeroed(t):
    return torch.where(t.isfinite(), t, torch.zeros_like(t))


def oracle_of(q, k, v, do, mask):
    return of.attention(zeroed(q).double(), zeroed(k).double(), zeroed(v).double(), q.shape[-1] ** -0.5, q.dtype, None,
                        mask, zeroed(do).double())


def some_mask(seed, *shape, share=0.6):
    return torch.rand(shape, generator=torch.Generator().manual_seed(seed)) < share


# queries, keys: more rows than 32 of several tiles of both sides; at most 32 rows per key head (the served form)
SHAPES = [(50, 130, 2, 1), (3, 300, 4, 1)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dim", [24, 40, 64, 80, 128])
@pytest.mark.parametrize("tq,tk,h,hk", SHAPES, ids=str)
def test_visible_bad_values(ctx, dtype, dim, tq, tk, h, hk):
    """v holds +inf, -inf and NaN at single elements: those columns of the queries that see them, no other."""
    banner(f"attention visible bad values {dtype} {dim} {tq} x {tk}")
    q, k, v, do = inputs(dim, 2, tq, tk, h, hk, dim, DTYPES[dtype])
    mask = some_mask(dim + 1, 2, h, tq, tk)
    mask[:, :, 1] = False
    v[0, 5, 0, 3], v[0, 70, 0, 17], v[1, tk - 2, 0, 9] = math.inf, -math.inf, math.nan
    v[1, 33, 0, 1], v[1, 35, 0, 1] = math.inf, -math.inf  # both seen: NaN
    check(run(ctx, q, k, v, do, mask), formulas(q, k, v, do, mask), oracle_of(q, k, v, do, mask))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dim", [24, 40, 64, 80, 128])
@pytest.mark.parametrize("tq,tk,h,hk", SHAPES, ids=str)
def test_visible_bad_gradients(ctx, dtype, dim, tq, tk, h, hk):
    """do holds infinities and NaN: dv is bad at that element alone (of the keys the query sees), their other gradients
    throughout."""
    banner(f"attention visible bad gradients {dtype} {dim} {tq} x {tk}")
    q, k, v, do = inputs(dim, 2, tq, tk, h, hk, dim, DTYPES[dtype])
    mask = some_mask(dim + 1, 2, h, tq, tk, share=0.3)
    mask[:, :, 1] = False
    do[0, 0, 0, 3], do[1, tq - 1, 1, 17], do[0, 2, 1, 5] = math.inf, math.nan, -math.inf
    do[1, 1, 0, 2] = math.inf  # of a query that sees nothing
    check(run(ctx, q, k, v, do, mask), formulas(q, k, v, do, mask), oracle_of(q, k, v, do, mask))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dim", [24, 64, 80, 128])
@pytest.mark.parametrize("tq,tk,h,hk", SHAPES, ids=str)
def test_visible_bad_queries_and_keys(ctx, dtype, dim, tq, tk, h, hk):
    """A NaN in q spoils its query and, of what its keys get, their gradients; a NaN in k every query that sees it."""
    banner(f"attention visible bad queries and keys {dtype} {dim} {tq} x {tk}")
    q, k, v, do = inputs(dim, 2, tq, tk, h, hk, dim, DTYPES[dtype])
    mask = some_mask(dim + 1, 2, h, tq, tk, share=0.3)
    mask[:, :, 1] = False
    mask[1, :, :, 40] = False
    mask[1, 0, 2, 40] = True
    q[0, 0, 0, 3], q[0, 1, 0, 1] = math.nan, math.inf  # the second sees nothing
    k[1, 40, 0, 5] = math.nan
    check(run(ctx, q, k, v, do, mask), formulas(q, k, v, do, mask), oracle_of(q, k, v, do, mask))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dim", [32, 96, 128])
def test_a_key_at_minus_infinity_is_a_weight_of_zero(ctx, dtype, dim):
    """k = inf where q < 0: the score is -inf, its weight 0; dq is NaN (0 inf) at that element alone."""
    banner(f"attention key at minus infinity {dtype} {dim}")
    q, k, v, do = inputs(dim, 1, 40, 100, 2, 1, dim, DTYPES[dtype])
    q[..., 7] = -q[..., 7].abs() - 0.1
    k[0, 50, 0, 7] = math.inf
    mask = some_mask(dim + 1, 1, 2, 40, 100)
    clean = of.attention(q.double(), zeroed(k).double(), v.double(), dim ** -0.5, q.dtype, None,
                         mask & (torch.arange(100) != 50), do.double())
    check(run(ctx, q, k, v, do, mask), formulas(q, k, v, do, mask), clean)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dim", [32, 96, 128])
@pytest.mark.parametrize("masked", [False, True])
def test_a_key_of_no_weight_gets_no_gradient(ctx, dtype, dim, masked):
    """k = inf where every query is negative: each weight is 0, and so are the key's dk and dv, also beside the rows past
    the last that fill up a tile."""
    banner(f"attention key of no weight {dtype} {dim} masked {masked}")
    q, k, v, do = inputs(dim, 1, 45, 100, 1, 1, dim, DTYPES[dtype])
    q[..., 7] = -q[..., 7].abs() - 0.1
    k[0, 50, 0, 7] = math.inf
    got = run(ctx, q, k, v, do, torch.ones((1, 1, 45, 100), dtype=torch.bool) if masked else None)
    assert (got["dk"][0, 50] == 0).all() and (got["dv"][0, 50] == 0).all()
    for name in ("o", "lse", "dk", "dv"):
        assert got[name].isfinite().all(), name


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("which", ["v", "do"])
def test_a_mask_that_shows_everything_is_no_mask(ctx, dtype, which):
    banner(f"attention all-true mask, bad {which} {dtype}")
    q, k, v, do = inputs(3, 1, 70, 90, 2, 1, 48, DTYPES[dtype])
    bad = v if which == "v" else do
    bad[0, 11, 0, 4], bad[0, 60, 0, 30], bad[0, 61, 0, 31] = math.inf, -math.inf, math.nan
    a = run(ctx, q, k, v, do, None)
    b = run(ctx, q, k, v, do, torch.ones((1, 1, 70, 90), dtype=torch.bool))
    for name in ("o", "lse", "dv"):
        assert torch.equal(a[name].isnan(), b[name].isnan()), name
        assert torch.equal(a[name][a[name].isinf()], b[name][b[name].isinf()]), name
    for name in ("dq", "dk"):
        assert torch.equal(a[name].isfinite(), b[name].isfinite()), name
