"""GPU cross attention where its tile pipelines turn: workgroups that stream many tiles of either side, few queries under
masks, and the bits that the score gradients keep. Against the fp64 oracle within its bounds."""
import math

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


def inputs(seed, b, tq, tk, h, hk, d, dtype):
    return (normal(seed, (b, tq, h, d), dtype), normal(seed + 1, (b, tk, hk, d), dtype),
            normal(seed + 2, (b, tk, hk, d), dtype), normal(seed + 3, (b, tq, h, d), dtype))


def some_mask(seed, *shape, share=0.5):
    return torch.rand(shape, generator=torch.Generator().manual_seed(seed)) < share


def run(ctx, q, k, v, do, lengths=None, mask=None):
    from differentiable_gaussian_splatting_amd import gsr
    q, k, v, do = (t.cuda() for t in (q, k, v, do))
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    mask = None if mask is None else mask.cuda()
    o, lse = gsr.gsr_cross_attention_forward(ctx, q, k, v, None, lens, mask)
    return (o, lse) + gsr.gsr_cross_attention_backward(ctx, q, k, v, o, lse, do, None, lens, mask)


def check(got, q, k, v, do, lengths=None, mask=None):
    want = of.attention(q.double(), k.double(), v.double(), q.shape[-1] ** -0.5, q.dtype, lengths, mask, do.double())
    for name, g in zip(("o", "lse", "dq", "dk", "dv"), got):
        within(g, want[name], want["e_" + name], name)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("h,dim", [(32, 32), (32, 40), (32, 64), (96, 64), (32, 80), (32, 128), (96, 128)])
def test_workgroups_that_stream_many_tiles(dtype, h, dim, masked):
    """512 workgroups of 128 rows in each kernel, which no rule has a reason to split, so each streams every tile: 4 to 8
    of 64 or 32 keys or rows (64 and 32 at most). That nothing was split is read off the scratch: a part of a split takes
    room in the arena, and the limit leaves none beside do.o of the rows. Lengths end inside tiles of either size."""
    from differentiable_gaussian_splatting_amd import gsr
    banner(f"attention many tiles {dtype} {h} heads of {dim} masked {masked}")
    tq = 250 if h == 32 else 84
    lengths = [250, 249, 97, 64, 33, 0, 161, 250]
    q, k, v, do = inputs(dim, 8, tq, 250, h, 32, dim, DTYPES[dtype])
    mask = some_mask(dim, 8, 1, tq, 250) if masked else None
    for b, n in enumerate(lengths):
        k[b, n:], v[b, n:] = math.nan, math.inf
    c = gsr.Context(0)
    try:
        gsr.gsr_set_option(c, gsr.GSR_OPT_ARENA_LIMIT, 4 * 8 * h * tq)
        got = run(c, q, k, v, do, lengths, mask)
        check(got, q, k, v, do, lengths, mask)
        for b, n in enumerate(lengths):
            assert (got[3][b, n:] == 0).all() and (got[4][b, n:] == 0).all()
    finally:
        c.close()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dim", [24, 64, 80, 128])
@pytest.mark.parametrize("tq,tk", [(1, 2), (1, 130), (7, 5), (7, 290), (1, 5000), (7, 5000)])
def test_few_queries_under_masks(ctx, dtype, dim, tq, tk):
    """At most 32 rows to a key head: short and long contexts, hidden keys that hold anything, a query that sees nothing,
    and (past 3,000 keys) a stretch that nobody sees, which leaves whole parts of split keys empty."""
    banner(f"attention few queries masked {dtype} {dim} {tq} x {tk}")
    q, k, v, do = inputs(dim + tq, 2, tq, tk, 4, 1, dim, DTYPES[dtype])
    mask = some_mask(dim, 2, 4, tq, tk)
    mask[0, :, :, tk // 2] = True
    mask[:, :, :, 3::10] = False
    if tk > 3000:
        mask[..., 900:3700] = False
        k[:, 1000:1200], v[:, 3000:3300] = math.nan, math.inf
    mask[1, 2, tq - 1] = False
    k[:, 3::20], v[:, 3::20], k[:, 13::20], v[:, 13::20] = math.nan, math.inf, -math.inf, math.nan
    q[1, tq - 1, 2], do[1, tq - 1, 2] = math.nan, math.inf
    got = run(ctx, q, k, v, do, mask=mask)
    check(got, q, k, v, do, mask=mask)
    assert (got[0][1, tq - 1, 2] == 0).all() and got[1][1, 2, tq - 1] == -math.inf
    check(run(ctx, q, k, v, do, [tk - tk // 3, tk], mask), q, k, v, do, [tk - tk // 3, tk], mask)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dim", [64, 128])
def test_few_queries_that_stream_many_tiles(dtype, dim):
    """256 key heads of one query group each: one workgroup a key head, which streams all of its tiles (no scratch)."""
    from differentiable_gaussian_splatting_amd import gsr
    banner(f"attention few queries, many tiles {dtype} {dim}")
    q, k, v, do = inputs(dim, 16, 1, 700, 64, 16, dim, DTYPES[dtype])
    mask = some_mask(dim, 16, 1, 1, 700)
    lengths = [700 - 43 * b for b in range(16)]
    c = gsr.Context(0)
    try:
        gsr.gsr_set_option(c, gsr.GSR_OPT_ARENA_LIMIT, 1)
        for lens, m in ((None, None), (lengths, None), (lengths, mask)):
            o, lse = gsr.gsr_cross_attention_forward(
                c, q.cuda(), k.cuda(), v.cuda(), None, None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda(),
                None if m is None else m.cuda())
            want = of.attention(q.double(), k.double(), v.double(), dim ** -0.5, q.dtype, lens, m)
            within(o, want["o"], want["e_o"], "o")
            within(lse, want["lse"], want["e_lse"], "lse")
    finally:
        c.close()


def coarse(seed, shape, dtype):
    """Normal values rounded to eighths: products of a few hundred of them are summed without rounding in float32."""
    return ((normal(seed, shape) * 8).round() / 8).to(dtype)


def bits_of_ds(dtype, dim, masked):
    """Inputs, the formulas' values with do.o = 0, and the bounds of dq and dk with ds kept to twice the type's bits: the
    scores and do.v are exact, so an element of ds has the rounding of the scaled score, of lse and of the exponential
    (float32, relative to the largest exponent) and of three products; then ds, the float32 sums of its products, and the
    result are rounded."""
    t, tq, tk = DTYPES[dtype], 24, 40
    q, k, v, do = (coarse(dim + i, (1, n, h, dim), t) for i, (n, h) in enumerate(((tq, 2), (tk, 1), (tk, 1), (tq, 2))))
    mask = some_mask(dim, 1, 2, tq, tk, share=0.7) if masked else None
    scale, u = dim ** -0.5, of.ROUND[t]
    want = score_gradients(q, k, v, do, scale, mask, lambda ds: ds)
    span = float((want["s"].masked_fill(want["p"] == 0, 0.0)).abs().max() + want["lse"].abs().max())
    terms = max(tk, 2 * tq)
    e_ds = ((4 * span + 24 + terms) * of.U32 + u * u) * want["ds"].abs()
    e_dq = (e_ds @ k.double().abs().transpose(1, 2)).transpose(1, 2)
    e_dk = (e_ds.transpose(-1, -2) @ q.double().abs().transpose(1, 2)).sum(1, keepdim=True).transpose(1, 2)
    return (q, k, v, do), mask, scale, want, {"dq": e_dq + u * want["dq"].abs() + of.TINY[t],
                                              "dk": e_dk + u * want["dk"].abs() + of.TINY[t]}


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128])
def test_score_gradients_keep_twice_the_bits(ctx, dtype, dim, masked):
    """dq and dk in 16 bits come from ds kept as the sum of two 16-bit values. The backward gets o = 0, which makes do.o
    exactly 0 and leaves no other 16-bit rounding in them but their own."""
    from differentiable_gaussian_splatting_amd import gsr
    banner(f"attention bits of ds {dtype} {dim} masked {masked}")
    (q, k, v, do), mask, scale, want, bounds = bits_of_ds(dtype, dim, masked)
    # one rounding of ds, in the oracle, is outside the bounds
    once = score_gradients(q, k, v, do, scale, mask, lambda ds: rounded(ds, q.dtype))
    for name in bounds:
        assert ((once[name] - want[name]).abs() > 2 * bounds[name]).any(), name
    m = None if mask is None else mask.cuda()
    zero = torch.zeros_like(q).cuda()
    q, k, v, do = (x.cuda() for x in (q, k, v, do))
    got = gsr.gsr_cross_attention_backward(ctx, q, k, v, zero, want["lse"].float().cuda(), do, scale, None, m)
    within(got[0], want["dq"], bounds["dq"], "dq")
    within(got[1], want["dk"], bounds["dk"], "dk")


def rounded(x, dtype):
    """x with one rounding to the type's number of bits, whatever its size."""
    e = 2.0 ** torch.floor(torch.log2(x.abs().clamp_min(1e-300)))
    return (x / e).to(dtype).double() * e


def score_gradients(q, k, v, do, scale, mask, keep):
    q, k, v, do = (t.double().transpose(1, 2) for t in (q, k, v, do))
    s = scale * q @ k.transpose(-1, -2)
    if mask is not None:
        s = s.masked_fill(~mask, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None])
    ds = keep(scale * p * (do @ v.transpose(-1, -2)))
    return {"s": s, "lse": lse, "p": p, "ds": ds, "dq": (ds @ k).transpose(1, 2),
            "dk": (ds.transpose(-1, -2) @ q).sum(1, keepdim=True).transpose(1, 2)}
