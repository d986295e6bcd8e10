"""The fp64 reference of the selective scan, the causal convolution and clipping:
hand-computed cases, and its gradients against central differences."""
import numpy as np
import pytest

from oracle import ssm_oracle as O


def _scan_inputs(rng, T=5, B=2, D=6, N=3, G=2):
    x = {n: rng.normal(size=(T, B, D)) for n in ("x", "dt", "z")}
    x["A"] = -np.exp(rng.normal(size=(D, N)))
    x["Bm"], x["Cm"] = rng.normal(size=(T, B, G, N)), rng.normal(size=(T, B, G, N))
    x["D"], x["dt_bias"] = rng.normal(size=D), rng.normal(size=D)
    x["h0"] = rng.normal(size=(B, D, N))
    return x


def test_scan_one_step_by_hand():
    y, h, _ = O.scan_forward(np.full((1, 1, 1), 2.0), np.full((1, 1, 1), 0.5), np.array([[-1.0, -2.0]]),
                             np.array([[[[1.0, 3.0]]]]), np.array([[[[4.0, 5.0]]]]), h0=np.array([[[1.0, 1.0]]]),
                             D=np.array([7.0]), softplus=False)
    want = np.exp([-0.5, -1.0]) + 0.5 * 2.0 * np.array([1.0, 3.0])
    assert np.allclose(h[0, 0], want)
    assert np.allclose(y[0, 0, 0], want @ [4.0, 5.0] + 14.0)


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("lengths", [None, [3, 0], [5, 1]])
def test_scan_gradients_are_differences(lengths, softplus):
    rng = np.random.default_rng(3)
    x = _scan_inputs(rng)
    dy, dh = rng.normal(size=x["x"].shape), rng.normal(size=x["h0"].shape)

    def loss(v):
        y, h, _ = O.scan_forward(**v, lengths=lengths, softplus=softplus)
        return (y * dy).sum() + (h * dh).sum()

    y, h, kept = O.scan_forward(**x, lengths=lengths, softplus=softplus)
    # steps of either sign without softplus: states grow, and the two losses are rounded at their terms' size
    terms = np.abs(y * dy).sum() + np.abs(h * dh).sum()
    back = {n: v for n, v in x.items() if n not in ("dt_bias", "h0")}
    g = O.scan_backward(dy, **back, kept=kept, dhT=dh, lengths=lengths, softplus=softplus)
    names = {"x": "dx", "dt": "ddt", "z": "dz", "A": "dA", "Bm": "dB", "Cm": "dC", "D": "dD", "dt_bias": "ddt_bias",
             "h0": "dh0"}
    eps = 1e-6
    for n, gn in names.items():
        d = rng.normal(size=x[n].shape)
        want = (loss({**x, n: x[n] + eps * d}) - loss({**x, n: x[n] - eps * d})) / (2 * eps)
        assert abs((g[gn] * d).sum() - want) <= 1e-6 * (1 + abs(want)) + 2.0 ** -50 * terms / eps, n


def test_conv_by_hand():
    x = np.array([1.0, 2.0, 3.0]).reshape(3, 1, 1)
    y, s, _ = O.conv_forward(x, np.array([[10.0, 1.0]]), np.array([0.5]), np.array([[[4.0]]]), silu=False)
    assert np.allclose(y.ravel(), [41.5, 12.5, 23.5]) and np.allclose(s.ravel(), [3.0])


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("lengths", [None, [1, 0], [6, 2]])
def test_conv_gradients_are_differences(lengths, silu):
    rng = np.random.default_rng(4)
    T, B, D, W = 6, 2, 3, 4
    v = {"x": rng.normal(size=(T, B, D)), "w": rng.normal(size=(D, W)), "bias": rng.normal(size=D),
         "s0": rng.normal(size=(B, W - 1, D))}
    dy, ds = rng.normal(size=(T, B, D)), rng.normal(size=(B, W - 1, D))

    def loss(v):
        y, s, _ = O.conv_forward(**v, lengths=lengths, silu=silu)
        return (y * dy).sum() + (s * ds).sum()

    g = O.conv_backward(dy, v["w"], O.conv_forward(**v, lengths=lengths, silu=silu)[2], ds, lengths, silu)
    eps = 1e-6
    for n, gn in {"x": "dx", "w": "dw", "bias": "dbias", "s0": "ds0"}.items():
        d = rng.normal(size=v[n].shape)
        want = (loss({**v, n: v[n] + eps * d}) - loss({**v, n: v[n] - eps * d})) / (2 * eps)
        assert abs((g[gn] * d).sum() - want) <= 1e-6 * (1 + abs(want)), n


def test_clip_by_hand():
    norm, out = O.clip([np.array([3.0]), np.array([[4.0]])], 1.0, 0.0)
    assert norm == 5.0 and np.allclose(out[0], 0.6) and np.allclose(out[1], 0.8)
    norm, out = O.clip([np.array([3.0, 4.0])], 10.0)
    assert np.array_equal(out[0], [3.0, 4.0])
    norm, out = O.clip([np.array([np.inf]), np.array([1.0])], 1.0)
    assert norm == np.inf and out[1][0] == 1.0
