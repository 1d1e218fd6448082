"""Helpers of the feature operators' GPU tests: seeded inputs in the tested type, and element-wise bounds."""
from __future__ import annotations

import torch

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def normal(seed, shape, dtype=torch.float32, scale=1.0):
    """Seeded normal values rounded to dtype, on the CPU."""
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, dtype=torch.float32)).to(dtype)


def within(got, want, bound, what):
    """Every element of `got` within `bound` of `want` (the same special values where want is not finite)."""
    got, want, bound = got.detach().cpu().double(), want.double(), bound.double().expand(want.shape)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if not got.numel():
        return
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine & ~want.isnan()], want[~fine & ~want.isnan()]), what
    assert torch.equal(got.isnan(), want.isnan()), what
    err = (got - want).abs()[fine]
    ratio = err / bound[fine].clamp_min(1e-300)
    worst = float(ratio.max()) if ratio.numel() else 0.0
    print(f"  {what}: worst error / bound {worst:.3g}", flush=True)
    assert worst <= 1.0, (what, worst, float(err.max()))
