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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,N", [(20, 8), (20, 16), (20, 40), (640, 16)])
def test_gradients_of_extreme_steps(T, N, dtype):
    """Channel by channel, in one piece and (640 tokens) in several segments."""
    import torch
    import bwd_persistent_cta_gb300 as R
    B, D = 2, 16
    t = _inputs(T, B, D, N, 1, dtype, 5)
    t["dt"][:, :, 0] = -200.0
    t["dt"][:, :, 1] = 300.0
    t["dt"][::2, :, 2] = 80.0
    t["z"][:, :, 3] = -300.0
    t["z"][:, :, 4] = 300.0
    t["A"][5] = 0.0
    t["A"][6] = -float("inf")
    t["A"][7] = -float("inf")
    t["dt"][::3, :, 7] = -300.0
    t["dt"][:, :, 8] = -80.0
    host = {n: _np(v) for n, v in t.items()}
    host["A"][6:8] = RESET
    dev = {n: v.cuda() for n, v in t.items()}
    op = R.SelectiveScan(B, T, D, N, dtype=dtype)
    args, kw = [dev[n] for n in ARGS], {n: dev[n] for n in ("z", "D", "dt_bias")}
    y, hT = op.forward(*args, **kw, h0=dev["h0"])
    d = op.backward(dev["dy"], *args, **kw, dhT=dev["dhT"])
    wy, wh, kept = O.scan_forward(*(host[n] for n in ARGS + ("z", "D", "dt_bias", "h0")))
    want = O.scan_backward(host["dy"], *(host[n] for n in ARGS), kept, host["z"], host["D"], host["dhT"])
    # a walk over T tokens where nothing is forgotten (channel 5): the tolerances are of 600
    slack = max(1.0, T / 600)
    for c in range(D):
        _close(y[..., c], wy[..., c], slack * OUT_TOL[dtype], f"y of channel {c}")
        _close(hT[:, c], wh[:, c], slack * STATE_TOL[dtype], f"state of channel {c}")
        for n in ("dx", "ddt", "dz"):
            _close(d[n][..., c], want[n][..., c], slack * OUT_TOL[dtype], f"{n} of channel {c}")
        for n, w in (("dA", want["dA"][c]), ("dh0", want["dh0"][:, c])):
            _close(d[n][c] if n == "dA" else d[n][:, c], w, slack * GRAD_TOL[dtype], f"{n} of channel {c}")
        # sums of one number a channel may cancel: against the size of what is added
        for n, terms in (("dD", host["dy"] * host["x"] * host["z"]), ("ddt_bias", want["ddt"])):
            got = d[n][c].item()
            assert np.isfinite(got) and abs(got - want[n][c]) <= slack * GRAD_TOL[dtype] * np.abs(terms[..., c]).sum() + 2.0 ** -100, (n, c)
    for n in ("dB", "dC"):
        _close(d[n], want[n], slack * OUT_TOL[dtype], n)
