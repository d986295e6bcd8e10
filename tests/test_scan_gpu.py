"""The selective scan on the GPU against the fp64 reference: lengths on both sides of
each tile, every width of state, groups, lengths, strides, states, and its refusals.

Tolerances (2-norm of the difference over that of the reference, per tensor),
derived before the first run.  A state is rounded and multiplied by a rounded decay
once a token: over T <= 600 tokens a walk of sqrt(T) * 3 * 2^-24 = 4.4e-6, and the
gradients run the walk once more: fp32 storage 5e-6 (y, states) and 1e-5 (gradients).
bf16 storage takes decays from an approximation that is 2e-8 low on average: over 600
tokens of full memory 1.2e-5; fp32 results (states, gradients of A, D and the bias)
2e-5, bf16 results 1.5 * 2^-9, their own rounding."""
import numpy as np
import pytest

from oracle import ssm_oracle as O

pytestmark = pytest.mark.gpu

STATE_TOL = {"f32": 5e-6, "bf16": 2e-5}
GRAD_TOL = {"f32": 1e-5, "bf16": 2e-5}
OUT_TOL = {"f32": 1e-5, "bf16": 1.5 * 2.0 ** -9}
SEQ = ("x", "dt", "z", "Bm", "Cm")


def _close(got, want, tol, what):
    got = got.double().cpu().numpy()
    assert got.shape == want.shape, what
    assert np.all(np.isfinite(got)), what
    n, d = np.linalg.norm(want), np.linalg.norm(got - want)
    # a result below the normal range of both types (2^-126) may come out as zero
    assert d <= tol * n + (np.any(want) and 2.0 ** -126 * want.size ** 0.5), f"{what}: {d / n if n else d:.2e} > {tol:.1e}"


def _inputs(T, B, D, N, G, dtype, seed, softplus=True):
    """fp64 arrays whose values the handle's types hold exactly: steps from 0.001 to 0.1, rates from 1 to N."""
    import torch
    gen = torch.Generator().manual_seed(seed)
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    rnd = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    d0 = torch.exp(torch.empty(D).uniform_(np.log(1e-3), np.log(0.1), generator=gen))
    t = {"x": rnd(T, B, D), "dt": 0.7 * rnd(T, B, D), "z": rnd(T, B, D), "Bm": rnd(T, B, G, N), "Cm": rnd(T, B, G, N)}
    if not softplus:
        t["dt"] = d0 * torch.exp(t["dt"])
    t = {n: v.to(td) for n, v in t.items()}
    t["dy"] = rnd(T, B, D).to(td)
    t["A"] = -torch.arange(1.0, N + 1) * torch.exp(0.2 * rnd(D, N))
    # without softplus the bias is a step itself: a negative one would let states grow without bound
    t["D"], t["dt_bias"] = 1 + 0.1 * rnd(D), d0 + torch.log(-torch.expm1(-d0)) if softplus else d0
    t["h0"], t["dhT"] = 0.3 * rnd(B, D, N), 0.1 * rnd(B, D, N)
    return t


def _np(t):
    return None if t is None else t.double().numpy()


def _place(t, bfirst, packed):
    """On the GPU, in the order of the handle; ``packed`` in wider rows of NaN, off by some elements."""
    import torch
    t = t.transpose(0, 1).contiguous() if bfirst else t
    if not packed:
        return t.cuda()
    flat = t.flatten(2)
    wide = torch.full(flat.shape[:2] + (flat.shape[2] + 24,), float("nan"), dtype=t.dtype)
    wide[..., 8:8 + flat.shape[2]] = flat
    return wide.cuda()[..., 8:8 + flat.shape[2]].unflatten(2, t.shape[2:])


def _odd(t, bfirst):
    """Rows that start at odd elements, as B and C may."""
    import torch
    t = t.transpose(0, 1).contiguous() if bfirst else t
    flat = t.flatten(2)
    wide = torch.full(flat.shape[:2] + (flat.shape[2] + 5,), float("nan"), dtype=t.dtype)
    wide[..., 3:3 + flat.shape[2]] = flat
    return wide.cuda()[..., 3:3 + flat.shape[2]].unflatten(2, t.shape[2:])


def run(T, B, D, N, G=1, dtype="bf16", lengths=None, bfirst=False, packed=False, state=True, softplus=True, z=True,
        skip=True, bias=True, train=True, seed=0, poison=False, check=True, slack=1):
    import torch
    import bwd_persistent_cta_gb300 as R
    t = _inputs(T, B, D, N, G, dtype, seed + T + D + N, softplus)
    for n, on in (("z", z), ("D", skip), ("dt_bias", bias), ("h0", state), ("dhT", state)):
        if not on:
            t[n] = None
    host = {n: _np(v) for n, v in t.items()}
    if poison:                                    # what lies behind the last token
        for n in SEQ + ("dy",):
            if t[n] is not None:
                for b, length in enumerate(lengths):
                    t[n][length:, b] = float("nan") if b % 2 else float("inf")
    dev = {n: None if v is None else (_odd(v, bfirst) if packed and n in ("Bm", "Cm") else
                                      _place(v, bfirst, packed and n != "dy") if n in SEQ + ("dy",) else v.cuda())
           for n, v in t.items()}
    op = R.SelectiveScan(B, T, D, N, groups=G, dtype=dtype, softplus=softplus, batch_first=bfirst)
    if lengths is not None:
        op.set_seq_lengths(lengths)
    args = [dev[n] for n in ("x", "dt", "A", "Bm", "Cm")]
    kw = {n: dev[n] for n in ("z", "D", "dt_bias")}
    y, hT = op.forward(*args, **kw, h0=dev["h0"], train=train)
    d = op.backward(dev["dy"], *args, **kw, dhT=dev["dhT"]) if train else {}
    torch.cuda.synchronize()
    if not check:
        return y, hT, d
    fwd = {n: host[n] for n in ("x", "dt", "A", "Bm", "Cm", "z", "D", "dt_bias", "h0")}
    wy, wh, kept = O.scan_forward(**fwd, lengths=lengths, softplus=softplus)
    order = lambda a: a.transpose(0, 1) if bfirst else a  # noqa: E731
    _close(order(y), wy, slack * OUT_TOL[dtype], "y")
    _close(hT, wh, slack * STATE_TOL[dtype], "hT")
    if train:
        want = O.scan_backward(host["dy"], *(host[n] for n in ("x", "dt", "A", "Bm", "Cm")), kept, host["z"], host["D"],
                               host["dhT"], lengths, softplus)
        for n in ("dx", "ddt", "dz", "dB", "dC"):
            assert (d[n] is None) == (n == "dz" and not z)
            if d[n] is not None:
                _close(order(d[n]), want[n], slack * OUT_TOL[dtype], n)
        for n, on in (("dA", True), ("dD", skip), ("ddt_bias", bias), ("dh0", True)):
            assert (d[n] is not None) == on
            if on:
                _close(d[n], want[n], slack * GRAD_TOL[dtype], n)
    if lengths is not None:
        for b, length in enumerate(lengths):
            for v in [y] + [d[n] for n in ("dx", "ddt", "dz", "dB", "dC") if d.get(n) is not None]:
                assert not order(v)[length:, b].any()
    return y, hT, d


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 32, 33, 100])
def test_lengths(T, dtype):
    run(T, 2, 40, 16, dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [8, 16, 24, 32, 40, 64])
@pytest.mark.parametrize("D", [8, 24, 136])
def test_widths(D, N, dtype):
    run(37, 2, D, N, dtype=dtype, bfirst=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G,D,N", [(2, 16, 16), (3, 72, 16), (2, 272, 8), (4, 32, 64), (5, 200, 32)])
def test_groups(G, D, N, dtype):
    run(20, 3, D, N, G, dtype=dtype, packed=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bfirst", [False, True])
@pytest.mark.parametrize("packed", [False, True])
def test_layouts(packed, bfirst, dtype):
    run(45, 3, 64, 16, dtype=dtype, bfirst=bfirst, packed=packed)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bfirst", [False, True])
@pytest.mark.parametrize("lengths", [[50, 0, 17], [1, 16, 49], [0, 0, 0], [33, 32, 31]])
def test_unequal_lengths(lengths, bfirst, dtype):
    """What lies behind the last token is not read: NaN and infinities there change nothing."""
    run(50, 3, 72, 16, dtype=dtype, lengths=lengths, bfirst=bfirst, poison=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("off", ["z", "skip", "bias", "state", "softplus"])
def test_parts(off, dtype):
    run(40, 2, 48, 16, dtype=dtype, **{off: False})
    run(40, 2, 48, 8, dtype=dtype, z=False, skip=False, bias=False, state=False, softplus=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_memory(dtype):
    run(600, 2, 64, 16, dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,lengths", [(128, [128, 1]), (257, [130, 257]), (400, [399, 0]), (513, [64, 512]), (600, [333, 65])])
def test_segments_side_by_side(T, lengths, dtype):
    """Long sequences of few channels run as several segments, some of them behind the last token."""
    run(T, 2, 24, 16, dtype=dtype, lengths=lengths, poison=True)
    run(T, 2, 40, 8, dtype=dtype, bfirst=True, packed=True, state=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [8, 16, 40])
def test_many_segments(N, dtype):
    """As many segments as the length allows, one sequence ending early.  Roundings of the decays add up
    over a state's memory, which is the sequence at most: 2200 tokens here, 600 in the other tests."""
    run(2200, 2, 16, N, dtype=dtype, lengths=[2200, 1300], poison=True, bfirst=True, slack=2200 / 600)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_state_in_place_over_segments(dtype):
    import torch
    import bwd_persistent_cta_gb300 as R
    T, B, D, N = 512, 2, 24, 16
    t = {n: v.cuda() for n, v in _inputs(T, B, D, N, 1, dtype, 12).items()}
    op = R.SelectiveScan(B, T, D, N, dtype=dtype)
    args = [t[n] for n in ("x", "dt", "A", "Bm", "Cm")]
    y, hT = op.forward(*args, h0=t["h0"], train=False)
    for _ in range(3):
        h = t["h0"].clone()
        y2, h2 = op.forward(*args, h0=h, hT=h, train=False)
        assert h2.data_ptr() == h.data_ptr() and torch.equal(y, y2) and torch.equal(hT, h2)


def test_training_and_inference_agree():
    import torch
    a = run(50, 2, 136, 16, train=False, check=False)
    b = run(50, 2, 136, 16, train=True, check=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_same_inputs_same_bits():
    import torch
    a, b = (run(70, 3, 264, 16, check=False) for _ in range(2))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for n in a[2]:
        assert torch.equal(a[2][n], b[2][n]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extreme_steps(dtype):
    """Steps that underflow, and that forget everything; gates far on both sides; rates of zero and minus infinity."""
    import torch
    import bwd_persistent_cta_gb300 as R
    T, B, D, N = 20, 1, 16, 8
    t = _inputs(T, B, D, N, 1, dtype, 5)
    t["dt"][:, :, 0] = -200.0
    t["dt"][:, :, 1] = 300.0
    t["dt"][::2, :, 2] = 80.0
    t["z"][:, :, 3] = -300.0
    t["z"][:, :, 4] = 300.0
    t["A"][5] = 0.0
    host = {n: _np(v) for n, v in t.items()}
    host["A"][6] = -1e30                           # a reset at every token; the reference has no infinity times zero
    t["A"][6] = -float("inf")
    dev = {n: v.cuda() for n, v in t.items()}
    op = R.SelectiveScan(B, T, D, N, dtype=dtype)
    args = [dev[n] for n in ("x", "dt", "A", "Bm", "Cm")]
    kw = {n: dev[n] for n in ("z", "D", "dt_bias")}
    y, hT = op.forward(*args, **kw, h0=dev["h0"])
    wy, wh, kept = O.scan_forward(*(host[n] for n in ("x", "dt", "A", "Bm", "Cm", "z", "D", "dt_bias", "h0")))
    for d in range(D):
        _close(y[:, :, d], wy[:, :, d], OUT_TOL[dtype], f"y of channel {d}")
        _close(hT[:, d], wh[:, d], STATE_TOL[dtype], f"state of channel {d}")


@pytest.mark.parametrize("at", [0, 13, 16, 40])
def test_a_bad_token_shows(at):
    """A NaN in a valid token reaches every later output of its channel, and no other channel or sequence."""
    import torch
    import bwd_persistent_cta_gb300 as R
    T, B, D, N = 45, 2, 40, 16
    t = _inputs(T, B, D, N, 1, "bf16", 6)
    t["x"][at, 1, 3] = float("nan")
    dev = {n: v.cuda() for n, v in t.items()}
    op = R.SelectiveScan(B, T, D, N)
    y, hT = op.forward(*(dev[n] for n in ("x", "dt", "A", "Bm", "Cm")), train=False)
    bad = torch.isnan(y).cpu()
    want = torch.zeros(T, B, D, dtype=torch.bool)
    want[at:, 1, 3] = True
    assert torch.equal(bad, want)
    assert torch.isnan(hT[1, 3]).all() and torch.isnan(hT).sum() == N


def test_state_in_place():
    import torch
    import bwd_persistent_cta_gb300 as R
    T, B, D, N = 33, 2, 72, 16
    t = {n: v.cuda() for n, v in _inputs(T, B, D, N, 1, "bf16", 7).items()}
    op = R.SelectiveScan(B, T, D, N)
    args = [t[n] for n in ("x", "dt", "A", "Bm", "Cm")]
    y, hT = op.forward(*args, h0=t["h0"])
    y2, h2 = op.forward(*args, h0=t["h0"], hT=t["h0"])
    assert h2.data_ptr() == t["h0"].data_ptr()
    assert torch.equal(y, y2) and torch.equal(hT, h2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 5])
@pytest.mark.parametrize("D,N,G", [(8, 8, 1), (40, 16, 1), (264, 24, 3), (64, 64, 2), (72, 32, 1)])
def test_step(D, N, G, T, dtype):
    """Tokens against a pool in any order of slots; sequences without a slot are zero and touch nothing."""
    import torch
    import bwd_persistent_cta_gb300 as R
    B, pool = 5, 9
    t = _inputs(T, B, D, N, G, dtype, 8)
    lengths = [T, 0, T, (T + 1) // 2, T]
    slots = [7, 2, 0, 4, -1]
    state = torch.randn(pool, D, N, generator=torch.Generator().manual_seed(9))
    h0 = torch.stack([state[max(s, 0)] for s in slots])
    op = R.SelectiveScan(B, T, D, N, groups=G, dtype=dtype, batch_first=True)
    op.set_seq_lengths(lengths)
    dev = {n: _odd(v, True) if n in ("Bm", "Cm") else _place(v, True, True) if n in SEQ else v.cuda() for n, v in t.items()}
    st = state.clone().cuda()
    y = op.step(*(dev[n] for n in ("x", "dt", "A", "Bm", "Cm")), st, z=dev["z"], D=dev["D"], dt_bias=dev["dt_bias"],
                slots=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    host = {n: _np(v) for n, v in t.items()}
    wy, wh, _ = O.scan_forward(*(host[n] for n in ("x", "dt", "A", "Bm", "Cm", "z", "D", "dt_bias")), _np(h0),
                               [n if s >= 0 else 0 for n, s in zip(lengths, slots)])
    _close(y.transpose(0, 1), wy, OUT_TOL[dtype], "y")
    want = _np(state)
    for b, s in enumerate(slots):
        if s >= 0:
            want[s] = wh[b]
    _close(st, want, STATE_TOL[dtype], "pool")
    untouched = [i for i in range(pool) if i not in slots] + [2]
    assert torch.equal(st[untouched].cpu(), state[untouched])
    out_of = torch.full((B,), pool, dtype=torch.int32, device="cuda")
    keep = st.clone()
    y = op.step(*(dev[n] for n in ("x", "dt", "A", "Bm", "Cm")), st, slots=out_of)
    assert not y.any() and torch.equal(st, keep)


def test_steps_continue_a_sequence():
    import torch
    import bwd_persistent_cta_gb300 as R
    T, B, D, N = 21, 2, 40, 16
    t = {n: v.cuda() for n, v in _inputs(T, B, D, N, 1, "f32", 10).items()}
    whole, part, one = (R.SelectiveScan(B, n, D, N, dtype="f32") for n in (T, T - 4, 1))
    kw = {n: t[n] for n in ("D", "dt_bias")}
    cut = lambda n, a, b: t[n][a:b].contiguous()  # noqa: E731
    seq = ("x", "dt", "Bm", "Cm")
    y, hT = whole.forward(t["x"], t["dt"], t["A"], t["Bm"], t["Cm"], z=t["z"], **kw)
    x, dt, Bm, Cm = (cut(n, 0, T - 4) for n in seq)
    _, st = part.forward(x, dt, t["A"], Bm, Cm, **kw, train=False)
    for i in range(T - 4, T):
        x, dt, Bm, Cm = (cut(n, i, i + 1) for n in seq)
        yi = one.step(x, dt, t["A"], Bm, Cm, st, z=cut("z", i, i + 1), **kw)
        _close(yi[0], y[i].double().cpu().numpy(), 5e-6, f"token {i}")
    _close(st, hT.double().cpu().numpy(), 5e-6, "state")


def test_gradients_wanted_one_by_one():
    """Each gradient alone is the one that comes with all the others."""
    import torch
    import bwd_persistent_cta_gb300 as R
    T, B, D, N = 20, 2, 40, 16
    t = {n: v.cuda() for n, v in _inputs(T, B, D, N, 1, "f32", 11).items()}
    op = R.SelectiveScan(B, T, D, N, dtype="f32")
    args = [t[n] for n in ("x", "dt", "A", "Bm", "Cm")]
    kw = {n: t[n] for n in ("z", "D", "dt_bias")}
    op.forward(*args, **kw)
    d = op.backward(t["dy"], *args, **kw)
    a = op._inputs(*args, **kw)
    for n, want in d.items():
        got = torch.full_like(want, float("nan"))
        rc = R.rnn_scan_backward(op.handle, a, t["dy"].data_ptr(), None, R.rnn_scan_grad_t(**{n: got.data_ptr()}),
                                 op.backward_workspace.data_ptr(), op.reserve.data_ptr())
        assert rc == R.RNN_OK
        torch.cuda.synchronize()
        assert torch.equal(got, want), n


def test_refusals():
    import torch
    import bwd_persistent_cta_gb300 as R
    T, B, D, N = 3, 2, 16, 8
    op = R.SelectiveScan(B, T, D, N)
    bad, ws = R.RNN_BAD_PARAM, R.RNN_BAD_WORKSPACE
    m = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    p = m.data_ptr()
    good = dict(x=p, dt=p, B=p, C=p, A=p)

    def fwd(h0=None, y=p + 4096, hT=None, reserve=None, **kw):
        return R.rnn_scan_forward(op.handle, R.rnn_scan_in_t(**{**good, **kw}), h0, y, hT, None, reserve)

    assert fwd() == R.RNN_OK
    for kw in (dict(x=None), dict(dt=None), dict(A=None), dict(B=None), dict(C=None), dict(y=None), dict(x=p + 2),
               dict(dt=p + 8), dict(z=p + 2), dict(A=p + 4), dict(D=p + 4), dict(dt_bias=p + 4), dict(B=p + 1),
               dict(C=p + 1), dict(h0=p + 4), dict(hT=p + 4), dict(y=p + 2), dict(x_row=8), dict(dt_row=20), dict(z_row=4),
               dict(B_row=7), dict(C_row=-8), dict(x_row=-16)):
        assert fwd(**kw) == bad, kw
    assert fwd(reserve=p + 4) == ws
    assert fwd(B=p + 2, C=p + 6, B_row=9, C_row=11) == R.RNN_OK

    def bwd(dy=p, dhT=None, work=p + 8192, reserve=p + 4096, grad=None, **kw):
        return R.rnn_scan_backward(op.handle, R.rnn_scan_in_t(**{**good, **kw}), dy, dhT,
                                   R.rnn_scan_grad_t(**(grad or {})), work, reserve)

    assert op.backward_workspace_bytes <= 32768
    for kw in (dict(dy=None), dict(dy=p + 2), dict(dhT=p + 4), dict(grad=dict(dx=p + 2)), dict(grad=dict(dz=p)),
               dict(grad=dict(dD=p)), dict(grad=dict(ddt_bias=p)), dict(grad=dict(dA=p + 4)), dict(x=None)):
        assert bwd(**kw) == bad, kw
    for kw in (dict(work=None), dict(work=p + 4), dict(reserve=None), dict(reserve=p + 4)):
        assert bwd(**kw) == ws, kw

    def step(state=p + 4096, n=2, slots=None, y=p + 16384, **kw):
        return R.rnn_scan_step(op.handle, R.rnn_scan_in_t(**{**good, **kw}), state, n, slots, y)

    assert step() == R.RNN_OK
    for kw in (dict(state=None), dict(n=-1), dict(slots=p + 2), dict(y=None), dict(state=p + 4), dict(y=p + 2), dict(x=None)):
        assert step(**kw) == bad, kw
    assert R.rnn_scan_set_seq_lengths(op.handle, [4, 0]) == bad and R.rnn_scan_set_seq_lengths(op.handle, [-1, 0]) == bad
    torch.cuda.synchronize()
