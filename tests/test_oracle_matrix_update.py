"""The fp64 oracles of layer norm and of the orthogonalised updates (oracle/features.py) against their meaning, automatic
differentiation and differences, and the entry points' refusals and layouts that need no device."""
import ctypes
import os
import subprocess

import pytest
import torch

from oracle import features as of

QUINTIC = (3.4445, -4.7750, 2.0315)


def rnd(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def test_layer_norm_and_its_gradients():
    x, g, b, dy = rnd(1, 9, 12), 1 + 0.3 * rnd(2, 12), rnd(3, 12), rnd(4, 9, 12)
    leaves = [t.clone().requires_grad_(True) for t in (x, g, b)]
    y = torch.nn.functional.layer_norm(leaves[0], (12,), leaves[1], leaves[2], 1e-5)
    got = of.layer_norm(x, g, b, 1e-5, dy)
    assert torch.allclose(got["y"], y.detach(), rtol=1e-12, atol=1e-12)
    assert torch.allclose(got["mean"], x.mean(1)) and got["rstd"].shape == (9,)
    for name, w in zip(("dx", "dgamma", "dbeta"), torch.autograd.grad(y, leaves, dy)):
        assert torch.allclose(got[name], w, rtol=1e-10, atol=1e-10), name
    for at in (0, 31, 107):
        hi, lo = x.clone(), x.clone()
        hi.view(-1)[at] += 1e-5
        lo.view(-1)[at] -= 1e-5
        num = float(((of.layer_norm(hi, g, b, 1e-5)["y"] - of.layer_norm(lo, g, b, 1e-5)["y"]) * dy).sum() / 2e-5)
        assert abs(num - float(got["dx"].view(-1)[at])) < 1e-7 * (1 + abs(num))


@pytest.mark.parametrize("m,n", [(1, 1), (7, 7), (5, 12), (12, 5)])
def test_newton_schulz_moves_singular_values_alone(m, n):
    g = rnd(m + n, m, n)
    for steps in ([QUINTIC] * 5, [(1.5, -0.5, 0.0)] * 8, [(2.0, -1.5, 0.5)] * 2 + [QUINTIC]):
        assert torch.allclose(of.newton_schulz(g, steps), of.newton_schulz_svd(g, steps), rtol=0, atol=1e-9)
        assert torch.allclose(of.newton_schulz(g, steps, 0.5), of.newton_schulz_svd(g, steps, 0.5), rtol=0, atol=1e-9)
    assert (of.newton_schulz(0 * g, [QUINTIC]) == 0).all()


@pytest.mark.parametrize("spread", [0, 2])
def test_the_size_of_rounded_left_factors_holds(spread):
    """newton_schulz_error against the steps with A and P rounded to float16 in float64 arithmetic."""
    u, _, v = torch.linalg.svd(rnd(1, 60, 90), full_matrices=False)
    g = (u * 10.0 ** (-spread * torch.arange(60) / 60)) @ v if spread else rnd(2, 60, 90)
    steps = [QUINTIC] * 5
    near = lambda t: (t * 2.0 ** 10).half().double() / 2.0 ** 10  # noqa: E731
    x = g / g.norm()
    for a, b, c in steps:
        gram = near(near(x) @ near(x).T)
        x = a * x + near(b * gram + c * (gram @ gram)) @ x
    err = float((x - of.newton_schulz(g, steps)).norm())
    size = of.newton_schulz_error(g, steps, 2.0 ** -11, True)
    assert 0.05 * size < err < size, (err, size)


def test_null_contexts_are_refused_without_a_device():
    from differentiable_gaussian_splatting_amd import gsr
    lib = gsr.load()
    ln, ns = gsr.gsr_layer_norm(), gsr.gsr_newton_schulz()
    assert lib.gsr_layer_norm_forward(None, None, ctypes.byref(ln), *[None] * 5) == gsr.GSR_EINVAL
    assert lib.gsr_layer_norm_backward(None, None, ctypes.byref(ln), *[None] * 7) == gsr.GSR_EINVAL
    assert lib.gsr_orthogonalize(None, None, ctypes.byref(ns), None, None) == gsr.GSR_EINVAL
    assert lib.gsr_muon_step(None, None, ctypes.byref(ns), None, None, None, 0.1, 0.9, 1, 1.0) == gsr.GSR_EINVAL


def test_struct_layouts_match_the_header(tmp_path):
    from differentiable_gaussian_splatting_amd import gsr
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "gsr.h"', "int main(void) {"]
    structs = [gsr.gsr_layer_norm, gsr.gsr_newton_schulz]
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
