"""The block norm on the GPU against the fp64 reference, every combination of
its parts, widths on both sides of each thread layout, strided rows.

Tolerances (2-norm of the difference over that of the reference, per tensor),
derived before the first run: fp32 storage 2e-6 (row sums of up to 8192 terms
in a tree: below 20 * 2^-24 = 1.2e-6); bf16 storage 1.5 * 2^-9 = 2.9e-3 (the
output's rounding alone); fp32 weight gradients 5e-6 (a CTA adds its rows one
after the other: sqrt(rows) * 2^-24 of the sum, rows below 2000 here)."""
import numpy as np
import pytest

from oracle import lm_oracle as O

pytestmark = pytest.mark.gpu

TOL = {"f32": 2e-6, "bf16": 1.5 * 2.0 ** -9}
WEIGHT_TOL = 5e-6


def _close(got, want, tol, what):
    assert np.all(np.isfinite(got)), what
    n, d = np.linalg.norm(want), np.linalg.norm(got - want)
    assert d <= tol * n if n else d == 0, f"{what}: {d / n if n else d:.2e} > {tol:.1e}"


def _data(rows, groups, cols, dtype, seed):
    import torch
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator().manual_seed(seed)
    width = groups * cols
    rnd = lambda *s: torch.randn(s, generator=gen).to(td)  # noqa: E731
    t = {n: rnd(rows, width) for n in ("y", "z", "x", "dx_out", "dn_out")}
    t["y"] = (t["y"].float() * torch.exp(torch.randn(rows, 1, generator=gen))).to(td)
    for n in ("w_in", "scale", "w_out"):
        t[n] = (1 + 0.3 * torch.randn(cols, generator=gen)).to(td)
    return t


def _case(rows, groups, cols, dtype, gate, norm_in, residual, norm_out, weights=True, wide=False, seed=0, only=None):
    import torch
    import bwd_persistent_cta_gb300 as R
    t = _data(rows, groups, cols, dtype, seed + rows + cols)
    use = {"y": True, "z": gate is not None, "x": residual, "w_in": norm_in and weights,
           "scale": residual and weights, "w_out": norm_out and weights, "dx_out": only != "dn", "dn_out": norm_out and only != "dx"}
    host = {n: x.double().numpy() if use[n] else None for n, x in t.items()}
    dev = {}
    for n, x in t.items():
        if not use[n]:
            dev[n] = None
        elif wide and n in ("y", "z", "x"):
            w = torch.full((rows, x.shape[1] + 24), float("nan"), dtype=x.dtype)
            w[:, 8:8 + x.shape[1]] = x
            dev[n] = w.cuda()[:, 8:8 + x.shape[1]]
        else:
            dev[n] = x.cuda()
    op = R.BlockNorm(rows, cols, groups=groups, dtype=dtype, norm_in=norm_in, gate=gate, residual=residual,
                     norm_out=norm_out, eps=1e-5)
    args = {n: dev[n] for n in ("z", "x", "w_in", "scale", "w_out")}
    x_out, n_out = op.forward(dev["y"], **args)
    grads = op.backward(dev["dx_out"], dev["dn_out"], dev["y"], **args)
    torch.cuda.synchronize()
    fold = lambda a: None if a is None else a.reshape(rows * groups, cols)  # noqa: E731
    h = {n: fold(a) if n in ("y", "z", "x", "dx_out", "dn_out") else a for n, a in host.items()}
    kw = {n: h[n] for n in ("x", "w_in", "scale", "w_out")}
    c, n, saved = O.norm_forward(h["y"], h["z"], **kw, gate=gate, norm_in=norm_in, norm_out=norm_out, eps=1e-5)
    want = O.norm_backward(h["dx_out"], h["dn_out"], h["y"], saved, **kw, norm_in=norm_in)
    get = lambda a: fold(a.double().cpu().numpy()) if a.dim() == 2 else a.double().cpu().numpy()  # noqa: E731
    _close(get(x_out), c, TOL[dtype], "x_out")
    assert (n_out is not None) == norm_out
    if norm_out:
        _close(get(n_out), n, TOL[dtype], "n_out")
    for name, g in grads.items():
        if g is None:
            continue
        _close(get(g), want[name], WEIGHT_TOL if g.dim() == 1 else TOL[dtype], name)
    assert (grads["dz"] is not None) == (gate is not None) and (grads["dx"] is not None) == residual
    return x_out, n_out, grads


WIDTHS = [8, 56, 64, 72, 128, 136, 256, 264, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096, 4104, 8192]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols", WIDTHS)
def test_widths(cols, dtype):
    _case(37, 1, cols, dtype, "silu", True, True, True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [None, "silu", "sigmoid"])
@pytest.mark.parametrize("norm_in", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("norm_out", [False, True])
def test_parts(dtype, gate, norm_in, residual, norm_out):
    for cols in (128, 1024):
        _case(19, 2, cols, dtype, gate, norm_in, residual, norm_out, wide=True)
        _case(700, 1, cols, dtype, gate, norm_in, residual, norm_out, weights=False)


@pytest.mark.parametrize("rows,groups", [(1, 1), (1, 5), (3, 7), (2500, 16), (5000, 1)])
def test_rows_and_groups(rows, groups):
    _case(rows, groups, 128, "bf16", "silu", True, False, False, wide=True)


def test_one_upstream_gradient():
    _case(50, 1, 512, "bf16", "silu", True, True, True, only="dx")
    _case(50, 1, 512, "bf16", "silu", True, True, True, only="dn")


def test_zero_and_extreme_rows():
    """A row of zeros normalises to zero; large and small rows keep their scale; gates far on both sides stay finite."""
    import torch
    import bwd_persistent_cta_gb300 as R
    cols = 256
    y = torch.randn(4, cols)
    y[0] = 0
    y[1] *= 1e15
    y[2] *= 1e-12
    z = torch.linspace(-3e4, 3e4, cols).repeat(4, 1)
    op = R.BlockNorm(4, cols, dtype="f32", gate="silu", norm_out=True, eps=1e-6)
    x_out, n_out = op.forward(y.cuda(), z=z.cuda())
    d = op.backward(torch.ones(4, cols, device="cuda"), None, y.cuda(), z=z.cuda())
    for t in (x_out, n_out, d["dy"], d["dz"]):
        assert torch.isfinite(t).all()
    assert torch.all(x_out[0] == 0) and torch.all(n_out[0] == 0)
    c, n, _ = O.norm_forward(y.double().numpy(), z.double().numpy(), gate="silu", norm_out=True)
    _close(x_out.double().cpu().numpy(), c, TOL["f32"], "x_out")


def test_in_place_residual_and_repeats():
    import torch
    t = _data(300, 1, 1024, "bf16", 9)
    import bwd_persistent_cta_gb300 as R
    op = R.BlockNorm(300, 1024, gate="silu", residual=True, norm_out=True)
    a = {n: t[n].cuda() for n in ("z", "x", "w_in", "scale", "w_out")}
    y = t["y"].cuda()
    x1, n1 = op.forward(y, **a)
    d1 = op.backward(t["dx_out"].cuda(), t["dn_out"].cuda(), y, **a)
    d2 = op.backward(t["dx_out"].cuda(), t["dn_out"].cuda(), y, **a)
    for n in d1:
        assert torch.equal(d1[n], d2[n]), n
    x2, n2 = op.forward(y, **a, x_out=a["x"])
    assert x2.data_ptr() == a["x"].data_ptr()
    assert torch.equal(x1, x2) and torch.equal(n1, n2)


def test_another_stream():
    import torch
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        _case(64, 1, 2048, "bf16", "silu", True, True, True)


def test_refusals():
    import torch
    import bwd_persistent_cta_gb300 as R
    op = R.BlockNorm(4, 64, gate="silu", residual=True, norm_out=True)
    bad = R.RNN_BAD_PARAM
    t = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(64, device="cuda")
    p = t.data_ptr()
    good = dict(y=p, z=p, x=p)

    def fwd(x_out=p, n_out=p, **kw):
        return R.rnn_norm_forward(op.handle, R.rnn_norm_in_t(**{**good, **kw}), x_out, n_out)

    assert fwd() == R.RNN_OK
    for kw in (dict(y=None), dict(z=None), dict(x=None), dict(y=p + 2), dict(z=p + 8), dict(y_row=56), dict(z_row=68),
               dict(x_row=-64), dict(w_in=p + 4), dict(x_out=None), dict(n_out=None), dict(x_out=p + 2)):
        assert fwd(**kw) == bad, kw

    def bwd(dx_out=p, dn_out=p, dy=p, dz=p, dx=p, dw_in=None, dscale=None, dw_out=None, ws=None):
        return R.rnn_norm_backward(op.handle, R.rnn_norm_in_t(**good), dx_out, dn_out, dy, dz, dx, dw_in, dscale,
                                   dw_out, ws)

    assert bwd() == R.RNN_OK
    assert bwd(dx_out=None, dn_out=None) == bad
    assert bwd(dy=p + 2) == bad
    assert bwd(dw_in=w.data_ptr()) == R.RNN_BAD_WORKSPACE
    plain = R.BlockNorm(4, 64)
    x = R.rnn_norm_in_t(y=p)
    assert R.rnn_norm_forward(plain.handle, x, p, None) == R.RNN_OK
    assert R.rnn_norm_forward(plain.handle, x, p, p) == bad
    for i in (1, 3, 4, 6, 7):                      # dn_out, dz, dx, dscale, dw_out of parts that are left out
        args = [p, None, p, None, None, None, None, None]
        args[i] = p
        assert R.rnn_norm_backward(plain.handle, x, *args, None) == bad, i
    torch.cuda.synchronize()
