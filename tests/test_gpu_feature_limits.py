"""The feature operators at their limits: counts that do not fit 32 bits, offsets and launches past them, alignment."""
import math

import pytest
import torch

from featurehelp import normal
from gpuhelp import banner

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    from differentiable_gaussian_splatting_amd import gsr
    c = gsr.Context(0)
    yield c
    c.close()


def overflow(f, *args, **kw):
    from differentiable_gaussian_splatting_amd import gsr
    with pytest.raises(gsr.GsrError) as e:
        f(*args, **kw)
    assert e.value.status == gsr.GSR_EOVERFLOW


@pytest.mark.parametrize("extra", [0, 5])
def test_counts_of_more_than_32_bits_are_refused(ctx, extra):
    """2^32 + 5 of something is not taken for 5 of it: broadcast views of small tensors, and small outputs."""
    from differentiable_gaussian_splatting_amd import gsr
    banner(f"feature counts of 2^32 + {extra}")
    n = (1 << 32) + extra
    x, small = torch.zeros((1, 1, 4), device="cuda"), torch.zeros((1, 4, 4), device="cuda")
    stats = torch.zeros((1, 2, 2), device="cuda")
    for shape in ((1, n, 4), (n, 1, 4)):
        overflow(gsr.gsr_group_norm_forward, ctx, x.expand(shape), None, None, 2, stats=stats)
        overflow(gsr.gsr_group_norm_backward, ctx, x.expand(shape), None, None, 2, stats, x.expand(shape))
    overflow(gsr.gsr_group_norm_forward, ctx, small, None, None, n + 2, y=small, stats=stats)
    overflow(gsr.gsr_group_norm_forward, ctx, small, None, None, 2, 1e-5, n + 1, y=small, stats=stats)
    one, pos = torch.zeros((1, 1, 1, 8), device="cuda"), torch.zeros((1, 1, 1), device="cuda")
    overflow(gsr.gsr_rotary_forward, ctx, one.expand(1, 1, n, 8), pos, [2])
    overflow(gsr.gsr_rotary_forward, ctx, one.expand(n, 1, 1, 8), pos, [2])
    overflow(gsr.gsr_rotary_backward, ctx, one, pos, [n + 2], dx=one.clone())
    overflow(gsr.gsr_rotary_forward, ctx, one, pos, [2], 100.0, n + 1, out=one.clone())
    kv = one.expand(1, 3, 1, 8)
    for shape in ((1, n, 1, 8), (1, 1, n, 8)):
        overflow(gsr.gsr_cross_attention_forward, ctx, one.expand(shape), kv, kv)
        lse = torch.zeros(1, device="cuda")
        overflow(gsr.gsr_cross_attention_backward, ctx, one.expand(shape), kv, kv, one.expand(shape), lse,
                 one.expand(shape))
    overflow(gsr.gsr_cross_attention_forward, ctx, one, one.expand(1, n, 1, 8), one.expand(1, n, 1, 8))


def test_heads_of_no_elements_are_refused(ctx):
    from differentiable_gaussian_splatting_amd import gsr
    banner("attention heads of no elements")
    q, kv = torch.zeros((1, 2, 1, 0), device="cuda"), torch.zeros((1, 3, 1, 0), device="cuda")
    with pytest.raises(gsr.GsrError) as e:
        gsr.gsr_cross_attention_forward(ctx, q, kv, kv)
    assert e.value.status == gsr.GSR_EINVAL


def test_statistics_at_any_float_alignment(ctx):
    from differentiable_gaussian_splatting_amd import gsr
    banner("group norm statistics off 8-byte boundaries")
    for p in (40, 9000):  # one launch, several
        x, dy = normal(1, (2, p, 24)).cuda(), normal(2, (2, p, 24)).cuda()
        y, stats = gsr.gsr_group_norm_forward(ctx, x, None, None, 4, 1e-5, 1)
        ref = gsr.gsr_group_norm_backward(ctx, x, None, None, 4, stats, dy, 1)
        odd = torch.full((2 * 4 * 2 + 2,), 7.0, device="cuda")
        at = odd[1:-1].view(2, 4, 2)
        y2, _ = gsr.gsr_group_norm_forward(ctx, x, None, None, 4, 1e-5, 1, stats=at)
        assert torch.equal(y, y2) and torch.equal(at, stats) and odd[0] == 7 and odd[-1] == 7
        got = gsr.gsr_group_norm_backward(ctx, x, None, None, 4, at, dy, 1)
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_statistics_past_32_bits(ctx):
    """More than 2^32 (image, group) pairs: every image's statistics in its own place. One value a group, so the mean is
    the value itself and the result 0."""
    from differentiable_gaussian_splatting_amd import gsr
    banner("group norm of 2^32 + 4 * 2^19 groups")
    n, c = (1 << 13) + 4, 1 << 19
    row = normal(1, (c,), torch.bfloat16).cuda()
    y, stats = gsr.gsr_group_norm_forward(ctx, row.expand(n, 1, c), None, None, c, 1.0)
    for i in (0, 1, 3, 4, 4096, n - 5, n - 4, n - 1):
        assert torch.equal(stats[i, :, 0], row.float()) and (stats[i, :, 1] == 1).all() and (y[i] == 0).all(), i
    del y, stats
    torch.cuda.empty_cache()  # 43 GB


def test_more_workgroups_than_one_dimension_of_a_launch(ctx):
    """2^24 + 64 key heads of one query each: more than 2^32 threads."""
    from differentiable_gaussian_splatting_amd import gsr
    banner("attention of 2^24 + 64 key heads")
    b, h, tk, d = (1 << 22) + 16, 4, 3, 8
    k, v = normal(1, (1, tk, h, d), torch.float16).cuda(), normal(2, (1, tk, h, d), torch.float16).cuda()
    q = normal(3, (64, 1, h, d), torch.float16).cuda()
    few = [t.expand(64, tk, h, d) for t in (k, v)]
    ref_o, ref_lse = gsr.gsr_cross_attention_forward(ctx, q, *few)
    ref = gsr.gsr_cross_attention_backward(ctx, q, *few, ref_o, ref_lse, q)
    many = q.repeat(b // 64 + 1, 1, 1, 1)[:b]
    kv = [t.expand(b, tk, h, d) for t in (k, v)]
    o, lse = gsr.gsr_cross_attention_forward(ctx, many, *kv)
    got = gsr.gsr_cross_attention_backward(ctx, many, *kv, o, lse, many)
    for x, want in ((o, ref_o), (lse, ref_lse)) + tuple(zip(got, ref)):
        whole = x[:b // 64 * 64].view(-1, 64, *x.shape[1:])
        assert (whole == want).all() and torch.equal(x[b // 64 * 64:], want[:b % 64])


def test_more_chunks_to_copy_than_one_dimension_of_a_launch():
    """2^28 + 40 keys off a 16-byte boundary, of which 2^32 + 640 chunks are copied to the scratch (64 GiB): one key seen
    2^28 times, whose value is a power of two, so that the output is exact."""
    from differentiable_gaussian_splatting_amd import gsr
    banner("attention of 2^28 + 40 unaligned keys")
    n, d = (1 << 28) + 40, 128
    c = gsr.Context(0)
    try:
        q = torch.full((1, 1, 1, d), 0.125, dtype=torch.bfloat16, device="cuda")
        k = torch.full((d + 1,), 0.25, dtype=torch.bfloat16, device="cuda")[1:].view(1, 1, 1, d).expand(1, n, 1, d)
        v = torch.full((1, 1, 1, d), 0.5, dtype=torch.bfloat16, device="cuda")
        v[..., ::2] = -4
        o, lse = gsr.gsr_cross_attention_forward(c, q, k, v.expand(1, n, 1, d), 1.0)
        assert torch.equal(o, v)
        assert abs(float(lse) - (128 / 32 + math.log(n))) < 1e-5
    finally:
        c.close()


def test_more_rotary_workgroups_than_one_dimension_of_a_launch(ctx):
    """2^28 + 40 tokens of 128 pairs, 16 to a workgroup, turned in place (137 GB)."""
    from differentiable_gaussian_splatting_amd import gsr
    banner("rotary of 2^28 + 40 tokens of 256")
    n, d = (1 << 28) + 40, 256
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < n * (2 * d + 4) + (8 << 30):
        pytest.skip("needs 146 GB of device memory")
    x = torch.ones((1, n, 1, d), dtype=torch.bfloat16, device="cuda")
    pos = (torch.arange(n, device="cuda", dtype=torch.int32) % 1000).float().view(1, n, 1)
    gsr.gsr_rotary_forward(ctx, x, pos, [d // 2], out=x)
    for at in (0, 12345, (1 << 27) - 7, (1 << 28) - 100, n - 100):
        part = slice(at, at + 100)
        want = gsr.gsr_rotary_forward(ctx, torch.ones((1, 100, 1, d), dtype=torch.bfloat16, device="cuda"),
                                      pos[:, part].contiguous(), [d // 2])
        assert torch.equal(x[:, part], want), at
    del x
    torch.cuda.empty_cache()
