"""The causal convolution on the GPU against the fp64 reference: every width, lengths
around the state and the stretches of tokens a thread walks, lengths, strides, states,
and its refusals.

Tolerances (2-norm of the difference over that of the reference, per tensor), derived
before the first run: fp32 storage 1e-6 (sums of up to five terms and a sigmoid, a few
times 2^-24 each); bf16 storage 1.5 * 2^-9, the result's own rounding; the fp32
gradients of w and bias 2e-6 (tokens are added one after another within a stretch and
then the stretches: a walk below sqrt(T B) * 2^-24 of the sum, plus bf16 storage's
approximate sigmoid, 2^-21).  States are copies: equal."""
import numpy as np
import pytest

from oracle import ssm_oracle as O
from tests.test_scan_gpu import _close, _np, _place

pytestmark = pytest.mark.gpu

TOL = {"f32": 1e-6, "bf16": 1.5 * 2.0 ** -9}
WEIGHT_TOL = 2e-6


def _inputs(T, B, D, W, dtype, seed):
    import torch
    gen = torch.Generator().manual_seed(seed)
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    rnd = lambda *s: torch.randn(s, generator=gen).to(td)  # noqa: E731
    return {"x": rnd(T, B, D), "dy": rnd(T, B, D), "w": rnd(D, W), "bias": rnd(D), "s0": rnd(B, W - 1, D),
            "dsT": rnd(B, W - 1, D)}


def run(T, B, D, W, dtype="bf16", lengths=None, bfirst=False, packed=False, act="silu", bias=True, state=True, poison=False,
        check=True):
    import torch
    import bwd_persistent_cta_gb300 as R
    t = _inputs(T, B, D, W, dtype, T + D + W)
    for n, on in (("bias", bias), ("s0", state), ("dsT", state)):
        if not on:
            t[n] = None
    host = {n: _np(v) for n, v in t.items()}
    if poison:
        for b, length in enumerate(lengths):
            t["x"][length:, b] = t["dy"][length:, b] = float("nan") if b % 2 else float("inf")
    dev = {n: None if v is None else _place(v, bfirst, packed and n == "x") if n in ("x", "dy") else v.cuda()
           for n, v in t.items()}
    op = R.CausalConv(B, T, D, W, dtype=dtype, act=act, batch_first=bfirst)
    if lengths is not None:
        op.set_seq_lengths(lengths)
    y, sT = op.forward(dev["x"], dev["w"], bias=dev["bias"], s0=dev["s0"])
    d = op.backward(dev["dy"], dev["x"], dev["w"], bias=dev["bias"], s0=dev["s0"], dsT=dev["dsT"])
    torch.cuda.synchronize()
    if not check:
        return y, sT, d
    order = lambda a: a.transpose(0, 1) if bfirst else a  # noqa: E731
    wy, ws, kept = O.conv_forward(host["x"], host["w"], host["bias"], host["s0"], lengths, act == "silu")
    want = O.conv_backward(host["dy"], host["w"], kept, host["dsT"], lengths, act == "silu")
    _close(order(y), wy, TOL[dtype], "y")
    assert np.array_equal(_np(sT.cpu()), ws)
    _close(order(d["dx"]), want["dx"], TOL[dtype], "dx")
    _close(d["ds0"], want["ds0"], TOL[dtype], "ds0")
    _close(d["dw"], want["dw"], WEIGHT_TOL, "dw")
    assert (d["dbias"] is not None) == bias
    if bias:
        _close(d["dbias"], want["dbias"], WEIGHT_TOL, "dbias")
    if lengths is not None:
        for b, length in enumerate(lengths):
            assert not order(y)[length:, b].any() and not order(d["dx"])[length:, b].any()
    return y, sT, d


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 31, 32, 33, 67, 200])
def test_lengths(T, W, dtype):
    run(T, 2, 40, W, dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [8, 16, 264, 1024, 1032, 2056])
def test_channels(D, dtype):
    run(40, 2, D, 4, dtype=dtype, bfirst=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bfirst", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_layouts(packed, bfirst, dtype):
    run(70, 3, 48, 4, dtype=dtype, bfirst=bfirst, packed=packed)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 4])
@pytest.mark.parametrize("lengths", [[70, 0, 33], [1, 2, 3], [0, 0, 0], [32, 64, 31], [34, 35, 66]])
def test_unequal_lengths(lengths, W, dtype):
    """What lies behind the last token is not read; a sequence shorter than the state keeps part of the old one."""
    run(70, 3, 48, W, dtype=dtype, lengths=lengths, poison=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [dict(act=None), dict(bias=False), dict(state=False), dict(act=None, bias=False, state=False)],
                         ids=str)
def test_parts(kw, dtype):
    run(50, 2, 48, 4, dtype=dtype, **kw)


def test_many_sequences():
    run(3, 300, 24, 4)
    run(130, 40, 16, 3, dtype="f32")


def test_same_inputs_same_bits():
    import torch
    a, b = (run(200, 5, 136, 4, check=False) for _ in range(2))
    assert torch.equal(a[0], b[0]) and all(torch.equal(a[2][n], b[2][n]) for n in a[2])


def test_state_in_place():
    import torch
    import bwd_persistent_cta_gb300 as R
    for T in (2, 40):
        t = {n: v.cuda() for n, v in _inputs(T, 3, 40, 4, "bf16", 3).items()}
        op = R.CausalConv(3, T, 40, 4)
        y, sT = op.forward(t["x"], t["w"], s0=t["s0"])
        y2, s2 = op.forward(t["x"], t["w"], s0=t["s0"], sT=t["s0"])
        assert s2.data_ptr() == t["s0"].data_ptr() and torch.equal(y, y2) and torch.equal(sT, s2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("T", [1, 2, 5])
@pytest.mark.parametrize("D", [8, 1048])
def test_step(D, T, W, dtype):
    import torch
    import bwd_persistent_cta_gb300 as R
    B, pool = 5, 8
    t = _inputs(T, B, D, W, dtype, 5)
    lengths, slots = [T, 0, T, (T + 1) // 2, T], [7, 2, 0, 4, 8]
    state = torch.randn(pool, W - 1, D, generator=torch.Generator().manual_seed(6)).to(t["x"].dtype)
    s0 = torch.stack([state[s % pool] for s in slots])
    op = R.CausalConv(B, T, D, W, dtype=dtype, batch_first=True)
    op.set_seq_lengths(lengths)
    st = state.clone().cuda()
    y = op.step(_place(t["x"], True, True), t["w"].cuda(), st, bias=t["bias"].cuda(),
                slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    wy, ws, _ = O.conv_forward(_np(t["x"]), _np(t["w"]), _np(t["bias"]), _np(s0),
                               [n if s < pool else 0 for n, s in zip(lengths, slots)])
    _close(y.transpose(0, 1), wy, TOL[dtype], "y")
    want = _np(state)
    for b, s in enumerate(slots):
        if s < pool:
            want[s] = ws[b]
    assert np.array_equal(_np(st.cpu()), want)


def test_steps_continue_a_sequence():
    import torch
    import bwd_persistent_cta_gb300 as R
    T, B, D, W = 12, 2, 40, 4
    t = {n: v.cuda() for n, v in _inputs(T, B, D, W, "f32", 8).items()}
    whole, part, one = (R.CausalConv(B, n, D, W, dtype="f32") for n in (T, 2, 1))
    y, sT = whole.forward(t["x"], t["w"])
    _, st = part.forward(t["x"][:2].contiguous(), t["w"])
    for i in range(2, T):
        yi = one.step(t["x"][i:i + 1].contiguous(), t["w"], st)
        assert torch.equal(yi[0], y[i])
    assert torch.equal(st, sT)


def test_refusals():
    import torch
    import bwd_persistent_cta_gb300 as R
    op = R.CausalConv(2, 3, 16, 4)
    bad = R.RNN_BAD_PARAM
    m = torch.zeros(1 << 14, dtype=torch.uint8, device="cuda")
    p = m.data_ptr()
    good = dict(x=p, w=p)

    def fwd(s0=None, y=p + 4096, sT=None, **kw):
        return R.rnn_conv_forward(op.handle, R.rnn_conv_in_t(**{**good, **kw}), s0, y, sT)

    assert fwd() == R.RNN_OK
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(x=p + 2), dict(w=p + 8), dict(bias=p + 2), dict(s0=p + 2),
               dict(sT=p + 2), dict(y=p + 2), dict(x_row=8), dict(x_row=20), dict(x_row=-16)):
        assert fwd(**kw) == bad, kw

    def bwd(dy=p, dsT=None, dx=p + 4096, dw=None, dbias=None, ds0=None, work=None, **kw):
        return R.rnn_conv_backward(op.handle, R.rnn_conv_in_t(**{**good, **kw}), None, dy, dsT, dx, dw, dbias, ds0, work)

    assert bwd() == R.RNN_OK
    for kw in (dict(dy=None), dict(dy=p + 2), dict(dx=p + 2), dict(dw=p + 4), dict(dbias=p), dict(dsT=p + 2),
               dict(ds0=p + 8), dict(x=None)):
        assert bwd(**kw) == bad, kw
    assert bwd(dw=p + 4096) == R.RNN_BAD_WORKSPACE
    assert bwd(dw=p + 4096, work=p + 4) == R.RNN_BAD_WORKSPACE

    def step(state=p + 4096, n=2, slots=None, y=p + 8192, **kw):
        return R.rnn_conv_step(op.handle, R.rnn_conv_in_t(**{**good, **kw}), state, n, slots, y)

    assert step() == R.RNN_OK
    for kw in (dict(state=None), dict(n=-1), dict(slots=p + 2), dict(y=None), dict(state=p + 2), dict(x=None)):
        assert step(**kw) == bad, kw
    torch.cuda.synchronize()
