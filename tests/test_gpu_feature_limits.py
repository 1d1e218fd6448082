"""The feature operators at their limits: counts that do not fit 32 bits, offsets and launches past them, alignment."""
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
