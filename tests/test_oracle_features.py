"""The fp64 oracles of the feature operators (oracle/features.py) against automatic differentiation of plain forward
definitions and against central differences, and the operators' refusals that need no device."""
import ctypes
import math

import pytest
import torch

from oracle import features as of

torch.set_default_dtype(torch.float32)


def rnd(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


@pytest.mark.parametrize("kind", ["none", "silu", "relu"])
def test_group_norm_gradients(kind):
    x, g, b, dy = rnd(1, 2, 7, 12), 1 + 0.3 * rnd(2, 12), rnd(3, 12), rnd(4, 2, 7, 12)
    leaves = [t.clone().requires_grad_(True) for t in (x, g, b)]
    y = torch.nn.functional.group_norm(leaves[0].transpose(1, 2), 4, leaves[1], leaves[2], 1e-5).transpose(1, 2)
    y = {"none": lambda t: t, "silu": torch.nn.functional.silu, "relu": torch.relu}[kind](y)
    want = torch.autograd.grad(y, leaves, dy)
    got = of.group_norm(x, g, b, 4, 1e-5, kind, dy)
    assert torch.allclose(got["y"], y.detach(), rtol=1e-12, atol=1e-12)
    for name, w in zip(("dx", "dgamma", "dbeta"), want):
        assert torch.allclose(got[name], w, rtol=1e-10, atol=1e-10), name


def central(f, x, dy, at, h=1e-5):
    a, b = x.clone(), x.clone()
    a.view(-1)[at] += h
    b.view(-1)[at] -= h
    return float(((f(a) - f(b)) * dy).sum() / (2 * h))


def test_group_norm_gradient_by_differences():
    x, g, b, dy = rnd(1, 2, 5, 6), rnd(2, 6), rnd(3, 6), rnd(4, 2, 5, 6)
    dx = of.group_norm(x, g, b, 3, 1e-5, "silu", dy)["dx"]
    for at in (0, 7, 31, 59):
        num = central(lambda t: of.group_norm(t, g, b, 3, 1e-5, "silu")["y"], x, dy, at)
        assert abs(num - float(dx.view(-1)[at])) < 1e-7 * (1 + abs(num))


@pytest.mark.parametrize("halves", [False, True])
def test_rotary_turns_back_and_keeps_lengths(halves):
    x, pos = rnd(1, 2, 5, 3, 20), 50 * rnd(2, 2, 5, 3)
    y, _ = of.rotary(x, pos, [3, 2, 4], 100.0, halves)
    z, _ = of.rotary(y, pos, [3, 2, 4], 100.0, halves, back=True)
    assert torch.allclose(z, x, rtol=1e-12, atol=1e-12)
    assert torch.equal(y[..., 18:], x[..., 18:])
    # the backward is the transpose: <y, w> = <x, back(w)>
    w = rnd(3, 2, 5, 3, 20)
    assert torch.allclose((y * w).sum(), (x * of.rotary(w, pos, [3, 2, 4], 100.0, halves, back=True)[0]).sum())


def test_rotary_of_one_pair_by_hand():
    x = torch.tensor([1.0, 0.0, 7.0], dtype=torch.float64).reshape(1, 1, 1, 3)
    y, _ = of.rotary(x, torch.tensor([[[math.pi / 2]]], dtype=torch.float64), [1], 10000.0, False)
    assert torch.allclose(y.flatten(), torch.tensor([0.0, 1.0, 7.0], dtype=torch.float64), atol=1e-15)


def test_attention_gradients_and_empty_rows():
    q, k, v, do = rnd(1, 2, 5, 4, 6), rnd(2, 2, 7, 2, 6), rnd(3, 2, 7, 2, 6), rnd(4, 2, 5, 4, 6)
    mask = torch.rand((2, 4, 5, 7), generator=torch.Generator().manual_seed(5)) < 0.6
    mask[1, 2, 3] = False
    got = of.attention(q, k, v, 0.4, torch.float32, [7, 4], mask, do)
    ql, kl, vl = (t.clone().requires_grad_(True) for t in (q, k, v))
    see = mask & (torch.arange(7) < torch.tensor([7, 4])[:, None, None, None])
    s = 0.4 * torch.einsum("bthd,bjhd->bhtj", ql, kl.repeat_interleave(2, 2))
    p = torch.softmax(s.masked_fill(~see, -1e300), -1) * see.any(-1, keepdim=True)
    o = torch.einsum("bhtj,bjhd->bthd", p, vl.repeat_interleave(2, 2))
    assert torch.allclose(got["o"], o.detach(), rtol=1e-12, atol=1e-12)
    for name, w in zip(("dq", "dk", "dv"), torch.autograd.grad(o, (ql, kl, vl), do)):
        assert torch.allclose(got[name], w, rtol=1e-10, atol=1e-12), name
    assert got["lse"][1, 2, 3] == -math.inf and (got["o"][1, 3, 2] == 0).all() and (got["dq"][1, 3, 2] == 0).all()
    for at in (0, 17, 83):
        num = central(lambda t: of.attention(q, t, v, 0.4, torch.float32, [7, 4], mask)["o"], k, do, at)
        assert abs(num - float(got["dk"].reshape(-1)[at])) < 1e-7 * (1 + abs(num))


def test_attention_of_one_visible_key_is_its_value():
    q, k, v = rnd(1, 1, 3, 1, 4), rnd(2, 1, 5, 1, 4), rnd(3, 1, 5, 1, 4)
    k[0, 0] = math.nan
    v[0, 0] = math.inf
    mask = torch.zeros((1, 1, 3, 5), dtype=torch.bool)
    mask[..., 2] = True
    got = of.attention(q, k, v, 1.0, torch.float32, None, mask)
    assert torch.allclose(got["o"][0, :, 0], v[0, 2, 0].expand(3, 4))


def test_null_contexts_are_refused_without_a_device():
    from differentiable_gaussian_splatting_amd import gsr
    lib = gsr.load()
    gn, ro, at = gsr.gsr_group_norm(), gsr.gsr_rotary(), gsr.gsr_attention()
    assert lib.gsr_group_norm_forward(None, None, ctypes.byref(gn), *[None] * 5) == gsr.GSR_EINVAL
    assert lib.gsr_group_norm_backward(None, None, ctypes.byref(gn), *[None] * 8) == gsr.GSR_EINVAL
    assert lib.gsr_rotary_forward(None, None, ctypes.byref(ro), None, None, None) == gsr.GSR_EINVAL
    assert lib.gsr_rotary_backward(None, None, ctypes.byref(ro), None, None, None) == gsr.GSR_EINVAL
    assert lib.gsr_cross_attention_forward(None, None, ctypes.byref(at), *[None] * 7) == gsr.GSR_EINVAL
    assert lib.gsr_cross_attention_backward(None, None, ctypes.byref(at), *[None] * 11) == gsr.GSR_EINVAL


def test_feature_struct_layouts_match_the_header(tmp_path):
    import os
    import subprocess

    from differentiable_gaussian_splatting_amd import gsr
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "gsr.h"', "int main(void) {"]
    structs = [gsr.gsr_group_norm, gsr.gsr_rotary, gsr.gsr_attention]
    for cls in structs:
        n = cls.__name__
        lines.append(f'  printf("{n} %zu\\n", sizeof({n}));')
        lines += [f'  printf("{n}.{f} %zu\\n", offsetof({n}, {f}));' for f, _ in cls._fields_]
    src, exe = tmp_path / "l.c", tmp_path / "l"
    src.write_text("\n".join(lines + ["  return 0;", "}"]))
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", inc, str(src), "-o", str(exe)], check=True)
    got = dict(ln.split() for ln in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
               .splitlines())
    for cls in structs:
        assert int(got[cls.__name__]) == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(got[f"{cls.__name__}.{f}"]) == getattr(cls, f).offset, f
