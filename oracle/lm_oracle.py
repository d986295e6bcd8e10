"""fp64 CPU reference of the gated delta rule and the block norm (test
infrastructure only): the definitions, one token after the other, and the
gradients of each step by the chain rule."""
import numpy as np


def _heads(x, n):
    return np.repeat(x, n, axis=1)


def _fold(x, n):
    return x.reshape(x.shape[0], x.shape[1] // n, n, -1).sum(2)


def delta_forward(q, k, v, g, beta, s0=None, lengths=None, scale=None):
    """q, k [T, B, Hk, Dk], v [T, B, Hv, Dv], g, beta [T, B, Hv] -> o, sT [B, Hv, Dv, Dk] and the saved
    (states before each token, e).  Tokens at t >= lengths[b] are masked."""
    T, B, Hk, Dk = q.shape
    Hv, Dv = v.shape[2:]
    n = Hv // Hk
    scale = Dk ** -0.5 if scale is None else scale
    S = np.zeros((B, Hv, Dv, Dk)) if s0 is None else np.array(s0, dtype=np.float64)
    o = np.zeros((T, B, Hv, Dv))
    kept = []
    for t in range(T):
        live = np.ones(B, bool) if lengths is None else t < np.asarray(lengths)
        L = live[:, None]
        kt, qt = (np.where(L[..., None], _heads(x[t], n), 0.0) for x in (k, q))
        vt, gt, bt = np.where(L[..., None], v[t], 0.0), np.where(L, g[t], 0.0), np.where(L, beta[t], 0.0)
        Sa = np.exp(gt)[..., None, None] * S
        e = vt - np.einsum("bhvk,bhk->bhv", Sa, kt)
        kept.append((S, e))
        S = Sa + (bt[..., None] * e)[..., None] * kt[:, :, None, :]
        o[t] = scale * np.einsum("bhvk,bhk->bhv", S, qt)
    return o, S, kept


def delta_backward(do, q, k, v, g, beta, sT, kept, dsT=None, lengths=None, scale=None):
    """(dq, dk, dv, dg, dbeta, ds0) from delta_forward's sT and saved states."""
    T, B, Hk, Dk = q.shape
    Hv, Dv = v.shape[2:]
    n = Hv // Hk
    scale = Dk ** -0.5 if scale is None else scale
    dS = np.zeros((B, Hv, Dv, Dk)) if dsT is None else np.array(dsT, dtype=np.float64)
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    dg, dbeta = np.zeros(g.shape), np.zeros(beta.shape)
    after = sT
    for t in reversed(range(T)):
        live = np.ones(B, bool) if lengths is None else t < np.asarray(lengths)
        L = live[:, None]
        kt, qt = (np.where(L[..., None], _heads(x[t], n), 0.0) for x in (k, q))
        gt, bt = np.where(L, g[t], 0.0), np.where(L, beta[t], 0.0)
        dot = scale * np.where(L[..., None], do[t], 0.0)
        S, e = kept[t]
        Sa = np.exp(gt)[..., None, None] * S
        dq[t] = _fold(np.einsum("bhvk,bhv->bhk", after, dot), n)
        dS = dS + dot[..., None] * qt[:, :, None, :]
        y = np.einsum("bhvk,bhk->bhv", dS, kt)                  # gradient of u = beta e
        de = bt[..., None] * y
        dkt = np.einsum("bhvk,bhv->bhk", dS, bt[..., None] * e) - np.einsum("bhvk,bhv->bhk", Sa, de)
        dk[t] = _fold(np.where(L[..., None], dkt, 0.0), n)
        dv[t] = de
        dbeta[t] = np.where(L, (y * e).sum(-1), 0.0)
        dS = dS - de[..., None] * kt[:, :, None, :]
        dg[t] = np.where(L, (dS * Sa).sum((-1, -2)), 0.0)
        dS = np.exp(gt)[..., None, None] * dS
        after = S
    return dq, dk, dv, dg, dbeta, dS


def _gate(z, gate):
    if gate is None:
        return 1.0, 0.0
    s = 1.0 / (1.0 + np.exp(-z))
    return (z * s, s * (1 + z * (1 - s))) if gate == "silu" else (s, s * (1 - s))


def norm_forward(y, z=None, x=None, w_in=None, scale=None, w_out=None, gate=None, norm_in=True, norm_out=False,
                 eps=1e-6):
    """Rows [M, cols] -> (x', n or None, saved)."""
    one = lambda w: 1.0 if w is None else w  # noqa: E731
    r1 = 1.0 / np.sqrt((y * y).mean(1, keepdims=True) + eps) if norm_in else np.ones((y.shape[0], 1))
    f, df = _gate(z, gate)
    yn = y * r1
    a = yn * one(w_in)
    b = a * f
    c = b if x is None else x + one(scale) * b
    r2 = 1.0 / np.sqrt((c * c).mean(1, keepdims=True) + eps)
    return c, c * r2 * one(w_out) if norm_out else None, (r1, yn, a, b, c, r2, f, df)


def norm_backward(dx_out, dn_out, y, saved, x=None, w_in=None, scale=None, w_out=None, norm_in=True):
    """dict of the gradients (dz is zero without a gate)."""
    one = lambda w: 1.0 if w is None else w  # noqa: E731
    r1, yn, a, b, c, r2, f, df = saved
    d = np.zeros_like(c) if dx_out is None else dx_out.copy()
    out = {"dw_out": np.zeros(c.shape[1])}
    if dn_out is not None:
        h = dn_out * one(w_out)
        out["dw_out"] = (dn_out * c * r2).sum(0)
        d = d + r2 * h - c * r2 ** 3 * (h * c).mean(1, keepdims=True)
    out["dx"], out["dscale"] = d, (d * b).sum(0)
    db = d if x is None else d * one(scale)
    out["dz"] = db * a * df
    da = db * f
    out["dw_in"] = (da * yn).sum(0)
    h = da * one(w_in)
    out["dy"] = r1 * h - y * r1 ** 3 * (h * y).mean(1, keepdims=True) if norm_in else h
    return out
