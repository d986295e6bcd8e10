"""The selective scan at the ends of its range: rates of minus infinity and zero, steps that
underflow or forget everything, gates far on both sides, through the sequences forward
and backward and through the serving step.  Tolerances as in test_scan_gpu.py, whose
walks are longer than the twenty tokens here."""
import numpy as np
import pytest

from oracle import ssm_oracle as O
from tests.test_scan_gpu import GRAD_TOL, OUT_TOL, STATE_TOL, _close, _inputs, _np

pytestmark = pytest.mark.gpu

ARGS = ("x", "dt", "A", "Bm", "Cm")
RESET = -1e30                  # the reference has no infinity times zero


def _never(T, B, D, N, dtype, softplus):
    """Channel 2: a reset at every token whose step is not zero; the steps of some tokens are."""
    t = _inputs(T, B, D, N, 1, dtype, 31, softplus)
    t["A"][2] = -float("inf")
    if not softplus:
        t["dt_bias"][2] = 0.0
    t["dt"][::2, :, 2] = -300.0 if softplus else 0.0
    t["dt"][0, :, 2] = 1.0 if softplus else 0.5
    return t


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 5])
@pytest.mark.parametrize("N", [8, 16, 40, 64])
def test_a_step_with_a_rate_of_minus_infinity(N, T, dtype, softplus):
    """What a prompt leaves in the pool, a step of zero keeps there, as a token of the prompt does."""
    import torch
    import bwd_persistent_cta_gb300 as R
    B, D = 2, 16
    t = _never(T, B, D, N, dtype, softplus)
    t["dt"][T - 1, :, 2] = -300.0 if softplus else 0.0
    host = {n: _np(v) for n, v in t.items()}
    host["A"][2] = RESET
    dev = {n: v.cuda() for n, v in t.items()}
    kw = {n: dev[n] for n in ("z", "D", "dt_bias")}
    args = [dev[n] for n in ARGS]
    wy, wh, _ = O.scan_forward(*(host[n] for n in ARGS + ("z", "D", "dt_bias", "h0")), softplus=softplus)
    op = R.SelectiveScan(B, T, D, N, dtype=dtype, softplus=softplus)
    st = dev["h0"].clone()
    y = op.step(*args, st, **kw)
    _close(y, wy, OUT_TOL[dtype], "y")
    _close(st, wh, STATE_TOL[dtype], "pool")
    yf, hT = op.forward(*args, **kw, h0=dev["h0"], train=False)
    _close(yf, wy, OUT_TOL[dtype], "y of the sequence")
    _close(hT, wh, STATE_TOL[dtype], "state of the sequence")
