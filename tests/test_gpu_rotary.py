"""GPU rotary positions against the fp64 oracle (oracle/features.py), element by element: the result's own rounding
plus the derived bound on the angle, the sine and cosine and the products."""
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


def grid(seed, b, t, axes, size=100.0):
    return size * torch.rand((b, t, axes), generator=torch.Generator().manual_seed(seed))


def check(ctx, x, pos, pairs, base, halves, xd=None):
    from differentiable_gaussian_splatting_amd import gsr
    xd = x.cuda() if xd is None else xd
    for back, fn in ((False, gsr.gsr_rotary_forward), (True, gsr.gsr_rotary_backward)):
        got = fn(ctx, xd, pos.cuda(), pairs, base, int(halves))
        want, e = of.rotary(x.double(), pos.double(), pairs, base, halves, back)
        within(got, want, e + of.ROUND[x.dtype] * (want.abs() + e) + of.TINY[x.dtype], "back" if back else "forward")
        rest = 2 * sum(pairs)
        assert torch.equal(got[..., rest:].cpu(), x[..., rest:])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("b,t,h,d,pairs", [
    (1, 1, 1, 2, [1]), (1, 1, 8, 64, [16, 16]), (2, 7, 3, 80, [10, 10, 10]), (1, 33, 5, 31, [4, 3]),
    (1, 9, 2, 20, [1, 2, 3, 4]), (1, 300, 16, 128, [16, 24, 24]), (2, 5, 1, 256, [128]), (1, 3, 2, 7, [0, 2]),
    (1, 3, 2, 6, [0]), (1, 2000, 24, 40, [20]), (1, 20000, 12, 64, [8, 8, 16])])
def test_sizes(ctx, dtype, halves, b, t, h, d, pairs):
    banner(f"rotary {dtype} halves {halves} {b}x{t}x{h}x{d} {pairs}")
    check(ctx, normal(t + d, (b, t, h, d), DTYPES[dtype]), grid(t, b, t, len(pairs)), pairs, 10000.0, halves)


def test_far_positions_keep_their_accuracy(ctx):
    banner("rotary far positions")
    x = normal(1, (1, 64, 2, 32))
    pos = torch.randint(-(1 << 24), 1 << 24, (1, 64, 2), generator=torch.Generator().manual_seed(2)).float()
    check(ctx, x, pos, [8, 8], 10000.0, False)


def test_shared_positions_strides_and_in_place(ctx):
    from differentiable_gaussian_splatting_amd import gsr
    banner("rotary strided")
    pos = grid(3, 1, 11, 2)
    x = normal(4, (3, 11, 4, 24), torch.bfloat16)
    check(ctx, x, pos, [6, 6], 100.0, False)
    packed = torch.zeros((3, 4, 11, 51), dtype=torch.bfloat16, device="cuda")
    view = packed.transpose(1, 2)[..., 1:25]  # heads before tokens, rows not 16-byte aligned
    view.copy_(x)
    check(ctx, x, pos, [6, 6], 100.0, False, view)
    check(ctx, x, pos, [6, 4], 100.0, True, view)
    want = gsr.gsr_rotary_forward(ctx, view, pos.cuda(), [6, 6], 100.0)
    gsr.gsr_rotary_forward(ctx, view, pos.cuda(), [6, 6], 100.0, out=view)
    assert torch.equal(view, want) and (packed[..., 25:] == 0).all() and (packed[..., 0] == 0).all()
    one = x[:, :1].cuda().expand(3, 11, 4, 24)  # the same features at every token
    got = gsr.gsr_rotary_forward(ctx, one, pos.cuda(), [6, 6], 100.0)
    ref = gsr.gsr_rotary_forward(ctx, one.contiguous(), pos.cuda(), [6, 6], 100.0)
    assert torch.equal(got, ref)


def test_special_values_stay_in_their_pair(ctx):
    from differentiable_gaussian_splatting_amd import gsr
    banner("rotary special values")
    x = normal(4, (1, 3, 2, 12))
    x[0, 1, 0, 4], x[0, 2, 1, 11] = float("nan"), float("inf")  # pair 2; the copied tail
    y = gsr.gsr_rotary_forward(ctx, x.cuda(), grid(1, 1, 3, 1).cuda(), [4]).cpu()
    hit = torch.zeros_like(x, dtype=torch.bool)
    hit[0, 1, 0, 4:6] = True
    assert torch.equal(y.isnan(), hit) and y[0, 2, 1, 11] == float("inf")


def test_other_stream_and_graph(ctx):
    from differentiable_gaussian_splatting_amd import gsr
    banner("rotary on another stream, in a graph")
    x, pos = normal(1, (2, 500, 6, 64), torch.float16).cuda(), grid(2, 2, 500, 2).cuda()
    ref = gsr.gsr_rotary_forward(ctx, x, pos, [16, 16])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = gsr.gsr_rotary_forward(ctx, x, pos, [16, 16], stream=s)
    s.synchronize()
    assert torch.equal(got, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gsr.gsr_rotary_forward(ctx, x, pos, [16, 16], out=got)
    for i in range(3):
        got.fill_(i)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, ref)


def test_refusals(ctx):
    from differentiable_gaussian_splatting_amd import gsr
    banner("rotary refusals")
    x, pos = torch.zeros((2, 5, 3, 16), device="cuda"), torch.zeros((2, 5, 2), device="cuda")
    f = lambda *a, **k: gsr.gsr_rotary_forward(ctx, *a, **k)  # noqa: E731
    for args in ((x, pos, [8, 1]), (x, pos, [4, 4], 0.0), (x, pos, [4, 4], float("inf")),
                 (x, pos, [4, 4], 100.0, 2)):
        with pytest.raises(gsr.GsrError) as e:
            f(*args)
        assert e.value.status == gsr.GSR_EINVAL
    with pytest.raises(ValueError):
        f(x, pos, [1] * 5)
    with pytest.raises(ValueError):
        f(x, pos, [8])
    with pytest.raises(ValueError):
        f(x, pos.expand(2, 5, 2)[:, :4], [4, 4])
    with pytest.raises(TypeError):
        f(x, pos.double(), [4, 4])
    with pytest.raises(TypeError):
        f(x.to(torch.int32), pos, [4, 4])
    with pytest.raises(ValueError):
        f(x.cpu(), pos, [4, 4])
    with pytest.raises(gsr.GsrError, match="overlap"):
        f(x, pos, [4, 4], out=torch.zeros((2, 5, 1, 16), device="cuda").expand(2, 5, 3, 16))
    lib = gsr.load()
    d = gsr.gsr_rotary(0, 1 << 16, 1 << 16, 1, 4, 0, 1)
    d.base = 10.0
    assert lib.gsr_rotary_forward(ctx.handle, None, ctypes.byref(d), None, None, None) == gsr.GSR_EOVERFLOW
    d = gsr.gsr_rotary(0, 1, 1, 1, 4, 0, 1)
    d.base = 10.0
    assert lib.gsr_rotary_forward(ctx.handle, None, ctypes.byref(d), None, None, None) == gsr.GSR_EINVAL
    assert f(x[:, :0], pos[:, :0].contiguous(), [4, 4]).shape == (2, 0, 3, 16)
