"""The fp64 references of the gated delta rule and the block norm against
central differences of their own forward passes: the gradient formulas are the
derivatives of the definitions."""
import numpy as np
import pytest

from oracle import lm_oracle as O

# central differences with step h of a function whose third derivative is of
# order one: truncation h^2 = 1e-10, rounding 1e-16 / h = 1e-11 of the value
H, TOL = 1e-5, 1e-7


def _diff(f, x, d):
    return (f(x + H * d) - f(x - H * d)) / (2 * H)


@pytest.mark.parametrize("lengths", [None, [5, 0, 3]])
@pytest.mark.parametrize("Hk,Hv", [(2, 2), (1, 3)])
def test_delta_gradients_are_derivatives(lengths, Hk, Hv):
    rng = np.random.default_rng(3)
    T, B, Dk, Dv = 5, 3, 8, 16
    q, k = rng.normal(size=(2, T, B, Hk, Dk)) / np.sqrt(Dk)
    v = rng.normal(size=(T, B, Hv, Dv))
    g, beta = -rng.uniform(0, 1, (T, B, Hv)), rng.uniform(0, 1, (T, B, Hv))
    s0, do, dsT = rng.normal(size=(B, Hv, Dv, Dk)), rng.normal(size=v.shape), rng.normal(size=(B, Hv, Dv, Dk))
    args = [q, k, v, g, beta, s0]
    o, sT, kept = O.delta_forward(*args, lengths=lengths)
    grads = O.delta_backward(do, *args[:5], sT, kept, dsT, lengths)
    for i, (x, dx) in enumerate(zip(args, grads)):
        d = rng.normal(size=x.shape)

        def loss(xi):
            o, s, _ = O.delta_forward(*args[:i], xi, *args[i + 1:], lengths=lengths)
            return (o * do).sum() + (s * dsT).sum()

        want, got = _diff(loss, x, d), (dx * d).sum()
        assert abs(got - want) <= TOL * max(1.0, np.linalg.norm(dx) * np.linalg.norm(d)), i


@pytest.mark.parametrize("gate", [None, "silu", "sigmoid"])
@pytest.mark.parametrize("norm_in,residual,norm_out", [(True, True, True), (True, False, False), (False, True, True),
                                                       (False, False, True)])
def test_norm_gradients_are_derivatives(gate, norm_in, residual, norm_out):
    rng = np.random.default_rng(4)
    M, N = 4, 16
    p = {"y": rng.normal(size=(M, N)), "z": rng.normal(size=(M, N)), "x": rng.normal(size=(M, N)),
         "w_in": rng.normal(size=N), "scale": rng.normal(size=N), "w_out": rng.normal(size=N)}
    if not residual:
        p["x"] = p["scale"] = None
    dx_out, dn_out = rng.normal(size=(M, N)), rng.normal(size=(M, N)) if norm_out else None
    if not norm_in:
        p["w_in"] = None
    if not norm_out:
        p["w_out"] = None

    def loss(**kw):
        c, n, _ = O.norm_forward(**{**p, **kw}, gate=gate, norm_in=norm_in, norm_out=norm_out)
        return (c * dx_out).sum() + ((n * dn_out).sum() if norm_out else 0.0)

    _, _, saved = O.norm_forward(**p, gate=gate, norm_in=norm_in, norm_out=norm_out)
    grads = O.norm_backward(dx_out, dn_out, p["y"], saved, p["x"], p["w_in"], p["scale"], p["w_out"], norm_in)
    for name, x in p.items():
        if x is None or (name == "z" and gate is None):
            continue
        d = rng.normal(size=x.shape)
        want, got = _diff(lambda xi: loss(**{name: xi}), x, d), (grads["d" + name] * d).sum()
        assert abs(got - want) <= TOL * max(1.0, np.linalg.norm(grads["d" + name]) * np.linalg.norm(d)), name


def test_delta_reset_and_masked_rows():
    """g = -inf forgets the state; a sequence without tokens passes its state through."""
    rng = np.random.default_rng(5)
    T, B, H, D = 4, 2, 1, 8
    q, k, v = rng.normal(size=(3, T, B, H, D))
    g, beta = np.full((T, B, H), -0.1), np.full((T, B, H), 0.5)
    g[2] = -np.inf
    s0 = rng.normal(size=(B, H, D, D))
    o, sT, _ = O.delta_forward(q, k, v, g, beta, s0, lengths=[4, 0])
    o2, s2, _ = O.delta_forward(q[2:], k[2:], v[2:], np.where(np.isinf(g[2:]), 0, g[2:]),
                                beta[2:], None, lengths=[2, 0])
    np.testing.assert_allclose(o[2:, 0], o2[:, 0])
    np.testing.assert_allclose(sT[0], s2[0])
    np.testing.assert_array_equal(sT[1], s0[1])
    np.testing.assert_array_equal(o[:, 1], 0)
