"""GPU cross attention, forward and backward, against the fp64 oracle (oracle/features.py), element by element within
the oracle's bounds: float32 sums and statistics, probabilities and score gradients rounded once to the tested type."""
import ctypes
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


def inputs(seed, b, tq, tk, h, hk, d, dtype, scale=1.0):
    return (normal(seed, (b, tq, h, d), dtype, scale), normal(seed + 1, (b, tk, hk, d), dtype, scale),
            normal(seed + 2, (b, tk, hk, d), dtype), normal(seed + 3, (b, tq, h, d), dtype))


def dev(t):
    return None if t is None else t.cuda()


def both(ctx, q, k, v, do, scale=None, lengths=None, mask=None, stream=None):
    from differentiable_gaussian_splatting_amd import gsr
    o, lse = gsr.gsr_cross_attention_forward(ctx, q, k, v, scale, lengths, mask, stream=stream)
    return (o, lse) + gsr.gsr_cross_attention_backward(ctx, q, k, v, o, lse, do, scale, lengths, mask, stream=stream)


def check(ctx, q, k, v, do, scale=None, lengths=None, mask=None, on_device=None):
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    dq, dk, dv, ddo = on_device or [t.cuda() for t in (q, k, v, do)]
    got = both(ctx, dq, dk, dv, ddo, scale, lens, dev(mask))
    want = of.attention(q.double(), k.double(), v.double(), scale or q.shape[-1] ** -0.5, q.dtype, lengths,
                        None if mask is None else mask != 0, do.double())
    for name, g in zip(("o", "lse", "dq", "dk", "dv"), got):
        within(g, want[name], want["e_" + name], name)
    return got


SIZES = [  # b, tq, tk, h, hk, d
    (1, 1, 1, 1, 1, 1), (1, 1, 33, 2, 1, 20), (2, 3, 31, 4, 2, 32), (1, 33, 64, 1, 1, 33), (1, 32, 65, 2, 2, 64),
    (1, 129, 127, 1, 1, 40), (2, 5, 300, 6, 3, 80), (1, 65, 129, 8, 1, 128), (1, 200, 7, 2, 1, 127), (1, 2, 700, 3, 3, 65),
    (1, 700, 2, 2, 2, 48), (3, 17, 96, 12, 4, 16)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_sizes(ctx, dtype, size):
    banner(f"attention {dtype} {size}")
    check(ctx, *inputs(sum(size), *size, DTYPES[dtype]))


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_few_queries_of_many_keys_are_split_and_joined(ctx, dtype):
    banner(f"attention split keys {dtype}")
    check(ctx, *inputs(5, 2, 1, 5000, 4, 2, 64, DTYPES[dtype]), lengths=[5000, 1733])


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_many_queries_of_few_keys(ctx, dtype):
    banner(f"attention split queries {dtype}")
    check(ctx, *inputs(6, 1, 3000, 5, 2, 1, 24, DTYPES[dtype]))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lengths", [[0, 1, 64, 150], [32, 33, 300, -5], [31, 149, 65, 0]])
def test_lengths(ctx, dtype, lengths):
    """Lengths of none, one and past the end (clamped); what lies beyond a length, NaN and infinities too, changes
    nothing, and gets gradients of 0."""
    banner(f"attention lengths {dtype} {lengths}")
    q, k, v, do = inputs(7, 4, 40, 150, 4, 2, 48, DTYPES[dtype])
    clamped = [min(max(n, 0), 150) for n in lengths]
    for b, n in enumerate(clamped):
        k[b, n:], v[b, n:] = math.nan, math.inf
    got = check(ctx, q, k, v, do, lengths=lengths)
    for b, n in enumerate(clamped):
        assert (got[3][b, n:] == 0).all() and (got[4][b, n:] == 0).all()
        if n == 0:
            assert (got[0][b] == 0).all() and (got[2][b] == 0).all() and (got[1][b] == -math.inf).all()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dim", [72, 96, 104, 128])
def test_wide_heads_of_several_tiles_with_lengths(ctx, dtype, dim):
    """Heads past 64 elements, whose backward keeps an operand in LDS: several tiles of queries and keys, lengths that end
    inside a tile, NaN and infinities beyond them."""
    banner(f"attention wide heads {dtype} {dim}")
    q, k, v, do = inputs(dim, 3, 300, 290, 4, 2, dim, DTYPES[dtype])
    lengths = [290, 0, 141]
    for b, n in enumerate(lengths):
        k[b, n:], v[b, n:] = math.nan, math.inf
    got = check(ctx, q, k, v, do, lengths=lengths)
    for b, n in enumerate(lengths):
        assert (got[3][b, n:] == 0).all() and (got[4][b, n:] == 0).all()


def some_mask(seed, *shape, share=0.5):
    return torch.rand(shape, generator=torch.Generator().manual_seed(seed)) < share


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", [(2, 6, 70, 131), (2, 1, 70, 131), (1, 1, 70, 131), (2, 1, 1, 131), (1, 6, 1, 131)],
                         ids=str)
def test_masks(ctx, dtype, shape):
    banner(f"attention mask {dtype} {shape}")
    mask = some_mask(8, *shape)
    mask[0, 0, :: 5] = False  # rows that see nothing
    mask[-1, -1, -1, :] = False
    mask[..., 37] = False  # and a key that nobody sees
    got = check(ctx, *inputs(9, 2, 70, 131, 6, 2, 40, DTYPES[dtype]), mask=mask)
    if shape[2] > 1:
        rows = ~mask.expand(2, 6, 70, 131).any(-1)
        assert (got[0].transpose(1, 2).cpu()[rows] == 0).all() and (got[1].cpu()[rows] == -math.inf).all()
        assert (got[2].transpose(1, 2).cpu()[rows] == 0).all()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("dim", [24, 128])
def test_what_is_masked_may_hold_anything(ctx, dtype, dim):
    """Keys, values and gradients that nothing looks at hold NaN and infinities, in the same tiles as visible ones, and
    each query sees another part of the keys."""
    banner(f"attention masked NaN {dtype} {dim}")
    q, k, v, do = inputs(11, 2, 50, 100, 2, 1, dim, DTYPES[dtype])
    mask = some_mask(12, 2, 2, 50, 100)
    mask[:, :, :, 3::10] = False
    mask[0, :, 7], mask[1, :, 20:30] = False, False
    k[:, 3::20], v[:, 3::20], k[:, 13::20], v[:, 13::20] = math.nan, math.inf, -math.inf, math.nan
    q[0, 7], do[0, 7], do[1, 20:30] = math.nan, math.inf, math.nan
    check(ctx, q, k, v, do, mask=mask)
    check(ctx, q, k, v, do, mask=mask, lengths=[100, 61])


def test_a_masked_pair_hides_a_bad_value_from_its_row_alone(ctx):
    """A value that is NaN reaches the queries that see it, and no other query of the same tile."""
    from differentiable_gaussian_splatting_amd import gsr
    banner("attention bad value seen by some")
    q, k, v, do = inputs(13, 1, 64, 40, 1, 1, 32, torch.bfloat16)
    mask = torch.ones((1, 1, 64, 40), dtype=torch.bool)
    mask[0, 0, ::2, 5] = False
    clean, _ = gsr.gsr_cross_attention_forward(ctx, q.cuda(), k.cuda(), v.cuda(), None, None, mask.cuda())
    v[0, 5, 0, 9] = math.nan
    o, _ = gsr.gsr_cross_attention_forward(ctx, q.cuda(), k.cuda(), v.cuda(), None, None, mask.cuda())
    hit = torch.zeros((1, 64, 1, 32), dtype=torch.bool)
    hit[0, 1::2, 0, 9] = True
    assert torch.equal(o.isnan().cpu(), hit)
    assert torch.equal(o[~hit.cuda()], clean[~hit.cuda()])


def test_bytes_other_than_one_are_visible(ctx):
    banner("attention uint8 mask")
    mask = (some_mask(14, 1, 1, 30, 70).to(torch.uint8) * torch.randint(1, 256, (1, 1, 30, 70))).to(torch.uint8)
    check(ctx, *inputs(15, 1, 30, 70, 2, 2, 16, torch.float32), mask=mask)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_large_and_small_scores(ctx, dtype):
    """Scores in the hundreds (one key takes all) and nearly equal scores over a long context, whose probabilities
    are below the smallest normal float16."""
    banner(f"attention score range {dtype}")
    check(ctx, *inputs(16, 1, 40, 90, 2, 1, 64, DTYPES[dtype], scale=6.0))
    check(ctx, *inputs(17, 1, 3, 9000, 1, 1, 32, DTYPES[dtype], scale=0.1))


def test_small_and_large_gradients_in_float16(ctx):
    """Upstream gradients of a mean loss (about 1e-4) and of a scaled one (about 1e4) keep their relative accuracy."""
    banner("attention float16 gradient range")
    for size in (1e-4, 1e4):
        q, k, v, do = inputs(18, 1, 70, 2000, 2, 1, 32, torch.float16)
        check(ctx, q, k, v, (do.float() * size).half(), scale=0.05)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_strides(ctx, dtype):
    """Heads before tokens, rows that are not 16-byte aligned, keys and values packed in one tensor, and keys of one
    scene broadcast over the batch."""
    banner(f"attention strides {dtype}")
    t = DTYPES[dtype]
    q, k, v, do = inputs(19, 2, 37, 70, 4, 2, 40, t)
    k = k[:1].expand(2, 70, 2, 40)
    qs = torch.zeros((2, 4, 37, 47), dtype=t, device="cuda").transpose(1, 2)[..., 3:43]
    qs.copy_(q)
    kv = torch.zeros((2, 70, 2, 2, 40), dtype=t, device="cuda")
    vs = kv[:, :, :, 1]
    vs.copy_(v)
    ks = k[:1].contiguous().cuda().expand(2, 70, 2, 40)
    dos = torch.zeros((37, 2, 4, 41), dtype=t, device="cuda").transpose(0, 1)[..., 1:]
    dos.copy_(do)
    check(ctx, q, k, v, do, on_device=(qs, ks, vs, dos))


def test_outputs_go_where_asked(ctx):
    from differentiable_gaussian_splatting_amd import gsr
    banner("attention output strides")
    q, k, v, do = (t.cuda() for t in inputs(20, 2, 21, 50, 4, 2, 24, torch.bfloat16))
    ref = both(ctx, q, k, v, do)
    big = [torch.full((t.shape[0], t.shape[2], t.shape[1], 31), 7.0, dtype=t.dtype, device="cuda")
           for t in (ref[0], ref[2], ref[3], ref[4])]
    o, dq, dk, dv = (t.transpose(1, 2)[..., 2:26] for t in big)
    _, lse = gsr.gsr_cross_attention_forward(ctx, q, k, v, out=o)
    gsr.gsr_cross_attention_backward(ctx, q, k, v, o, lse, do, dq=dq, dk=dk, dv=dv)
    for got, want, all_of in zip((o, dq, dk, dv), (ref[0], ref[2], ref[3], ref[4]), big):
        assert torch.equal(got, want)
        assert (all_of[..., :2] == 7).all() and (all_of[..., 26:] == 7).all()
    assert torch.equal(lse, ref[1])


def test_offsets_past_32_bits(ctx):
    """Keys and values whose elements lie further apart than 2^32."""
    from differentiable_gaussian_splatting_amd import gsr
    banner("attention offsets past 32 bits")
    q, k, v, do = inputs(21, 1, 9, 70, 1, 1, 16, torch.bfloat16)
    step = 1 << 26
    flat = torch.empty(69 * step + 64, dtype=torch.bfloat16, device="cuda")
    kf, vf = flat.as_strided((1, 70, 1, 16), (0, step, 16, 1)), flat[32:].as_strided((1, 70, 1, 16), (0, step, 16, 1))
    kf.copy_(k)
    vf.copy_(v)
    got = check(ctx, q, k, v, do, on_device=(q.cuda(), kf, vf, do.cuda()))
    o, lse = gsr.gsr_cross_attention_forward(ctx, q.cuda(), k.cuda(), v.cuda())
    assert torch.equal(o, got[0]) and torch.equal(lse, got[1])


def test_the_same_bits_again_and_on_another_stream(ctx):
    banner("attention repeats")
    for size in ((2, 300, 200, 4, 2, 64), (1, 1, 4000, 4, 1, 128), (1, 3000, 40, 2, 1, 40)):
        q, k, v, do = (t.cuda() for t in inputs(22, *size, torch.bfloat16))
        ref = both(ctx, q, k, v, do)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        for _ in range(3):
            got = both(ctx, q, k, v, do, stream=s)
            s.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(ref, got))


def test_graph_replays(ctx):
    from differentiable_gaussian_splatting_amd import gsr
    banner("attention in a graph")
    q, k, v, do = (t.cuda() for t in inputs(23, 1, 20, 3000, 4, 2, 64, torch.float16))
    ref = [t.clone() for t in both(ctx, q, k, v, do)]
    bufs = [torch.empty_like(t) for t in ref]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gsr.gsr_cross_attention_forward(ctx, q, k, v, out=bufs[0], lse=bufs[1])
        gsr.gsr_cross_attention_backward(ctx, q, k, v, bufs[0], bufs[1], do, dq=bufs[2], dk=bufs[3], dv=bufs[4])
    for i in range(3):
        for b in bufs:
            b.fill_(float(i))
        both(ctx, q[:, :5].contiguous(), k, v, do[:, :5].contiguous())
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, bufs)), i


def test_nothing_to_attend_to_or_from(ctx):
    banner("attention of nothing")
    for t in DTYPES.values():
        got = both(ctx, *(x.cuda() for x in inputs(24, 2, 5, 0, 4, 2, 16, t)))
        assert (got[0] == 0).all() and (got[1] == -math.inf).all() and (got[2] == 0).all()
        got = both(ctx, *(x.cuda() for x in inputs(24, 2, 0, 5, 4, 2, 16, t)))
        assert got[0].shape == (2, 0, 4, 16) and (got[3] == 0).all() and (got[4] == 0).all()
        got = both(ctx, *(x.cuda() for x in inputs(24, 0, 3, 5, 4, 2, 16, t)))
        assert got[3].shape == (0, 5, 2, 16)


def test_gradient_by_differences(ctx):
    """The gradients predict how a float32 result changes: central differences of <o, do> along a random direction,
    whose rounding noise is about 2^-24 * 1e3 / h and whose truncation is of order h^2."""
    from differentiable_gaussian_splatting_amd import gsr
    banner("attention gradient by differences")
    q, k, v, do = (t.cuda() for t in inputs(25, 1, 60, 90, 4, 2, 32, torch.float32))
    mask = some_mask(26, 1, 1, 60, 90).cuda()
    _, _, dq, dk, dv = both(ctx, q, k, v, do, mask=mask)
    h = 2.0 ** -7
    for at, (x, grad) in enumerate(((q, dq), (k, dk), (v, dv))):
        w = normal(27 + at, x.shape).cuda()
        w = w / w.norm()
        side = []
        for sign in (1, -1):
            args = [q, k, v]
            args[at] = x + sign * h * w
            o, _ = gsr.gsr_cross_attention_forward(ctx, *args, None, None, mask)
            side.append(float((o.double() * do.double()).sum()))
        num, want = (side[0] - side[1]) / (2 * h), float((grad.double() * w.double()).sum())
        # noise: o's errors (below 4e-6 of values up to 1, 7,680 of them, of both signs) times do, over h
        assert abs(num - want) <= 2e-3 + 1e-2 * abs(want), (at, num, want)


def test_refusals(ctx):
    from differentiable_gaussian_splatting_amd import gsr
    banner("attention refusals")
    q, k, v, do = (t.cuda() for t in inputs(28, 2, 6, 9, 4, 2, 16, torch.float32))
    f = lambda *a, **kw: gsr.gsr_cross_attention_forward(ctx, *a, **kw)  # noqa: E731
    for args in ((q, k, v, 0.0), (q, k, v, -1.0), (q, k, v, math.inf), (q, k, v, math.nan),
                 (q[:, :, :3], k, v), (torch.zeros((2, 6, 4, 136), device="cuda"),) + 2 * (
                     torch.zeros((2, 9, 2, 136), device="cuda"),)):
        with pytest.raises(gsr.GsrError) as e:
            f(*args)
        assert e.value.status == gsr.GSR_EINVAL
    with pytest.raises(gsr.GsrError, match="overlap"):
        f(q, k, v, out=torch.zeros((1, 6, 4, 16), device="cuda").expand(2, 6, 4, 16))
    o, lse = f(q, k, v)
    with pytest.raises(gsr.GsrError, match="overlap"):
        gsr.gsr_cross_attention_backward(ctx, q, k, v, o, lse, do, dk=torch.zeros_like(k[:1]).expand(2, 9, 2, 16))
    for bad in ((q, k[:, :8], v), (q, k, v[..., :8]), (q[0], k, v), (q.cpu(), k, v), (q.transpose(2, 3), k, v)):
        with pytest.raises(ValueError):
            f(*bad)
    with pytest.raises(TypeError):
        f(q.half(), k, v)
    with pytest.raises(TypeError):
        f(q.double(), k.double(), v.double())
    ones = torch.ones((2, 4, 6, 9), dtype=torch.bool, device="cuda")
    for kw in ({"mask": ones[:, :3]}, {"mask": ones[..., :8]}, {"mask": ones.transpose(2, 3)},
               {"mask": ones.cpu()}, {"kv_lengths": torch.ones(3, dtype=torch.int32, device="cuda")}):
        with pytest.raises(ValueError):
            f(q, k, v, **kw)
    with pytest.raises(TypeError):
        f(q, k, v, mask=ones.float())
    with pytest.raises(TypeError):
        f(q, k, v, kv_lengths=torch.ones(2, dtype=torch.int64, device="cuda"))
    lib = gsr.load()
    d = gsr.gsr_attention(0, 1 << 16, 16, 16, 1 << 12, 4, 16, 1.0)
    assert lib.gsr_cross_attention_forward(ctx.handle, None, ctypes.byref(d), *[None] * 7) == gsr.GSR_EOVERFLOW
    d = gsr.gsr_attention(0, 1, 1, 1, 4, 4, 16, 1.0)
    assert lib.gsr_cross_attention_forward(ctx.handle, None, ctypes.byref(d), *[None] * 7) == gsr.GSR_EINVAL
    assert lib.gsr_cross_attention_backward(ctx.handle, None, ctypes.byref(d), *[None] * 11) == gsr.GSR_EINVAL


def test_an_arena_limit_is_an_error_and_leaves_the_context_usable():
    from differentiable_gaussian_splatting_amd import gsr
    banner("attention under an arena limit")
    c = gsr.Context(0)
    try:
        gsr.gsr_set_option(c, gsr.GSR_OPT_ARENA_LIMIT, 1 << 17)
        q, k, v, _ = (t.cuda() for t in inputs(29, 4, 8, 6000, 8, 4, 128, torch.float32))
        with pytest.raises(gsr.GsrError) as e:
            gsr.gsr_cross_attention_forward(c, q, k, v)
        assert e.value.status == gsr.GSR_ENOMEM
        gsr.gsr_set_option(c, gsr.GSR_OPT_ARENA_LIMIT, 0)
        gsr.gsr_set_option(c, gsr.GSR_OPT_KERNEL_TIMING, 4)
        gsr.gsr_cross_attention_forward(c, q, k, v)
        assert len(gsr.gsr_kernel_times(c, gsr.GSR_STAGE_ATTENTION_FORWARD)) == 1
    finally:
        c.close()
