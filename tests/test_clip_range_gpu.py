"""Clipping where the norm or the factor leaves fp32: finite gradients whose norm does not
fit, and limits so far below the norm that the factor is below the smallest normal number.

Tolerances as in test_clip_gpu.py (2^-22 of a scaled fp32 value, 2^-8 in bf16), and half
a step of the smallest numbers of the type twice, where two products are rounded there."""
import numpy as np
import pytest

from oracle import ssm_oracle as O

pytestmark = pytest.mark.gpu


def _check(host, types, limit, inplace, eps=0.0):
    import torch
    import bwd_persistent_cta_gb300 as R
    td = {"f32": torch.float32, "bf16": torch.bfloat16}
    t = [torch.from_numpy(h).to(td[d]).cuda() for h, d in zip(host, types)]
    vals = [v.double().cpu().numpy() for v in t]
    assert all(np.isfinite(v).all() for v in vals)
    norm, want = O.clip(vals, limit, eps)
    out = None if inplace else [torch.full_like(v, float("nan")) for v in t]
    got = R.GradClip([v.numel() for v in t], types).clip(t, limit, eps=eps, out=out).item()
    most = float(np.finfo(np.float32).max)
    assert got == float("inf") if norm > most * (1 + 2.0 ** -20) else abs(got - norm) <= 2.0 ** -22 * norm
    for v, w, d in zip(t if inplace else out, want, types):
        tol, least = (2.0 ** -22, 2.0 ** -149) if d == "f32" else (2.0 ** -8, 2.0 ** -133)
        assert np.all(np.abs(v.double().cpu().numpy() - w) <= tol * np.abs(w) + least)


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("limit", [1.0, 1e-3, 1e20, 3e38])
def test_norm_beyond_fp32(limit, inplace):
    rng = np.random.default_rng(1)
    big = 1e38 * np.sign(rng.normal(size=100)) * rng.uniform(0.5, 3, size=100)
    _check([big, rng.normal(size=5000), 1e37 * rng.normal(size=77)], ["f32", "f32", "bf16"], limit, inplace)


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("scale,limit", [(1e36, 1e-3), (1e38, 1e-6), (1e38, 1e-30), (1e30, 1e-12), (1e20, 1e-42), (1.0, 1e-42)])
def test_factor_below_the_normal_numbers(scale, limit, inplace):
    rng = np.random.default_rng(2)
    limit = float(np.float32(limit))
    host = [scale * rng.uniform(-1, 1, size=3000), scale * rng.uniform(-1, 1, size=900), 1e-3 * scale * rng.normal(size=40)]
    _check(host, ["f32", "bf16", "f32"], limit, inplace)


def test_limits_at_the_norm():
    """A norm on the limit changes nothing; one step above it does."""
    import torch
    import bwd_persistent_cta_gb300 as R
    op = R.GradClip([2])
    for m, changed in ((5.0, False), (float(np.nextafter(np.float32(5), np.float32(0))), True)):
        g = torch.tensor([3.0, 4.0], device="cuda")
        assert op.clip([g], m, eps=0.0).item() == 5.0
        assert (g.tolist() != [3.0, 4.0]) == changed
