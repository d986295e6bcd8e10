"""fp64 CPU reference of the selective scan, the causal convolution and gradient
clipping (test infrastructure only): the definitions, one token after the other, and
the gradients of each step by the chain rule."""
import numpy as np


def _sigma(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def _softplus(v):
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def _spread(x, D):
    """[B, G, N] to every channel of its group."""
    return np.repeat(x, D // x.shape[1], axis=1)


def _live(t, B, lengths):
    return (np.ones(B, bool) if lengths is None else t < np.asarray(lengths))[:, None]


def scan_forward(x, dt, A, Bm, Cm, z=None, D=None, dt_bias=None, h0=None, lengths=None, softplus=True):
    """x, dt, z [T, B, D], A [D, N], Bm, Cm [T, B, G, N] -> y, hT [B, D, N] and what scan_backward takes.  Tokens at
    t >= lengths[b] are masked."""
    T, B, ch = x.shape
    h = np.zeros((B,) + A.shape) if h0 is None else np.array(h0, dtype=np.float64)
    y, kept = np.zeros(x.shape), []
    for t in range(T):
        L = _live(t, B, lengths)
        xt, raw = np.where(L, x[t], 0.0), np.where(L, dt[t], 0.0) + (0.0 if dt_bias is None else dt_bias)
        d = np.where(L, _softplus(raw) if softplus else raw, 0.0)
        Bt, Ct = (np.where(L[..., None], _spread(m[t], ch), 0.0) for m in (Bm, Cm))
        a = np.exp(np.where(L[..., None], d[..., None] * A, 0.0))
        before = h
        h = a * h + (d * xt)[..., None] * Bt
        yt = (Ct * h).sum(-1) + (0.0 if D is None else D * xt)
        kept.append((before, h, a, d, raw, yt))
        zt = None if z is None else np.where(L, z[t], 0.0)
        y[t] = np.where(L, yt if z is None else yt * zt * _sigma(zt), 0.0)
    return y, h, kept


def scan_backward(dy, x, dt, A, Bm, Cm, kept, z=None, D=None, dhT=None, lengths=None, softplus=True):
    """A dict of all gradients from scan_forward's saved values."""
    T, B, ch = x.shape
    G = Bm.shape[2]
    g = np.zeros((B,) + A.shape) if dhT is None else np.array(dhT, dtype=np.float64)
    out = {n: np.zeros(s.shape) for n, s in (("dx", x), ("ddt", x), ("dz", x), ("dB", Bm), ("dC", Cm), ("dA", A))}
    out["dD"], out["ddt_bias"] = np.zeros(ch), np.zeros(ch)
    fold = lambda v: v.reshape(B, G, ch // G, -1).sum(2)  # noqa: E731
    for t in reversed(range(T)):
        L = _live(t, B, lengths)
        before, h, a, d, raw, yt = kept[t]
        xt, do = np.where(L, x[t], 0.0), np.where(L, dy[t], 0.0)
        Bt, Ct = (np.where(L[..., None], _spread(m[t], ch), 0.0) for m in (Bm, Cm))
        if z is not None:
            zt = np.where(L, z[t], 0.0)
            s = _sigma(zt)
            out["dz"][t] = do * yt * s * (1 + zt * (1 - s))
            do = do * zt * s
        out["dC"][t] = fold(do[..., None] * h)
        g = g + do[..., None] * Ct
        out["dB"][t] = fold(g * (d * xt)[..., None])
        gB = (g * Bt).sum(-1)
        out["dx"][t] = np.where(L, d * gB + (0.0 if D is None else D * do), 0.0)
        p = g * a * before
        dd = np.where(L, xt * gB + (p * A).sum(-1), 0.0)
        out["dA"] += np.where(L[..., None], p * d[..., None], 0.0).sum(0)
        out["ddt"][t] = dd * _sigma(raw) if softplus else dd
        out["dD"] += (do * xt).sum(0)
        out["ddt_bias"] += out["ddt"][t].sum(0)
        g = np.where(L[..., None], a * g, g)
    out["dh0"] = g
    return out


def conv_forward(x, w, bias=None, s0=None, lengths=None, silu=True):
    """x [T, B, D], w [D, W], s0 [B, W - 1, D] -> y, sT and what conv_backward takes."""
    T, B, ch = x.shape
    W = w.shape[1]
    past = np.zeros((B, W - 1, ch)) if s0 is None else np.array(s0, dtype=np.float64)
    y, kept = np.zeros(x.shape), []
    for t in range(T):
        L = _live(t, B, lengths)
        row = np.concatenate([past, np.where(L, x[t], 0.0)[:, None]], 1)
        pre = np.einsum("bkd,dk->bd", row, w) + (0.0 if bias is None else bias)
        y[t] = np.where(L, pre * _sigma(pre) if silu else pre, 0.0)
        kept.append((row, pre))
        past = np.where(L[..., None], row[:, 1:], past)
    return y, past, kept


def conv_backward(dy, w, kept, dsT=None, lengths=None, silu=True):
    """A dict of the gradients dx, dw, dbias, ds0 from conv_forward's saved values."""
    T, B, ch = dy.shape
    W = w.shape[1]
    dpast = np.zeros((B, W - 1, ch)) if dsT is None else np.array(dsT, dtype=np.float64)
    dx, dw, dbias = np.zeros(dy.shape), np.zeros(w.shape), np.zeros(ch)
    for t in reversed(range(T)):
        L = _live(t, B, lengths)
        row, pre = kept[t]
        s = _sigma(pre)
        dp = np.where(L, dy[t] * (s * (1 + pre * (1 - s)) if silu else 1.0), 0.0)
        dw += np.einsum("bd,bkd->dk", dp, row)
        dbias += dp.sum(0)
        drow = np.einsum("bd,dk->bkd", dp, w)
        drow[:, 1:] += np.where(L[..., None], dpast, 0.0)
        dx[t] = drow[:, -1]
        # past of token t: all of the row but its own input, or (masked) what came after it
        dpast = np.where(L[..., None], np.concatenate([drow[:, :1], drow[:, 1:-1]], 1), dpast)
        dx[t] = np.where(L, dx[t], 0.0)
    return {"dx": dx, "dw": dw, "dbias": dbias, "ds0": dpast}


def clip(tensors, max_norm, eps=1e-6):
    """The norm of all tensors together and the scaled tensors."""
    norm = np.sqrt(sum(np.sum(np.square(t.astype(np.float64))) for t in tensors))
    factor = max_norm / (norm + eps) if np.isfinite(norm) and norm + eps > max_norm else 1.0
    return norm, [t * factor for t in tensors]
