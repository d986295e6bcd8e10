"""The gated delta rule on the GPU, through the C ABI, against the fp64
reference: both directions and the serving step, at the lengths, widths, masks
and layouts where chunks, slices and reductions can go wrong.

Tolerances (2-norm of the difference over the 2-norm of the reference, per
tensor), derived before the first run:
  * fp32 storage: 1e-5.  Sums of up to 256 products in fp32 carry
    sqrt(256) * 2^-24 = 1e-6 at most, and a value passes a handful of such sums.
  * bf16 storage: 3 * 2^-9 = 5.9e-3.  The output's own rounding is at most 2^-9,
    and no value passes more than one rounding to bf16 on its way (two terms of a
    sum rounded independently add in quadrature, below a second 2^-9).
  * fp32 states with bf16 storage: 5e-5.  A state's operands are held as pairs of
    bf16, good to 2^-17; four products on a value's way with up to three
    neglected terms each stay below 12 * 2^-18 = 4.6e-5."""
import numpy as np
import pytest

from oracle import lm_oracle as O

pytestmark = pytest.mark.gpu

TOL = {"f32": 1e-5, "bf16": 3 * 2.0 ** -9}
STATE_TOL = {"f32": 1e-5, "bf16": 5e-5}


def _torch():
    import torch
    return torch


def _inputs(T, B, Hk, Hv, Dk, Dv, dtype, seed, gate=1.0, k_common=0.3):
    """Seq-major inputs rounded to the storage type, as fp64 arrays: unit keys with a common component, decays of a few to
    a thousand tokens, states as a running sequence leaves them."""
    torch = _torch()
    rng = np.random.default_rng(seed)

    def unit(x):
        return x / np.linalg.norm(x, axis=-1, keepdims=True)

    td = torch.bfloat16 if dtype == "bf16" else torch.float32

    def rnd(x):
        return torch.from_numpy(np.ascontiguousarray(x)).to(td).double().numpy()

    q = rnd(unit(rng.normal(size=(T, B, Hk, Dk))))
    k = rnd(unit(rng.normal(size=(T, B, Hk, Dk)) + k_common))
    v = rnd(rng.normal(size=(T, B, Hv, Dv)))
    rate = gate * np.exp(rng.uniform(np.log(1e-3), np.log(0.5), size=Hv))
    g = rnd(-rate * rng.uniform(0.2, 2.0, size=(T, B, Hv)))
    beta = rnd(rng.uniform(0.0, 1.0, size=(T, B, Hv)))
    s0 = rng.normal(size=(B, Hv, Dv, Dk)).astype(np.float32) * 0.3
    do = rnd(rng.normal(size=(T, B, Hv, Dv)))
    dsT = rng.normal(size=(B, Hv, Dv, Dk)).astype(np.float32) * 0.1
    return dict(q=q, k=k, v=v, g=g, beta=beta, s0=s0, do=do, dsT=dsT)


def _dev(x, dtype, bfirst=False, packed=False, fill=None):
    """Device tensor of a seq-major array; ``packed``: a slice of rows three times as wide, the rest NaN."""
    torch = _torch()
    td = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    t = torch.from_numpy(np.ascontiguousarray(x)).to(td)
    if bfirst:
        t = t.transpose(0, 1).contiguous()
    if packed:
        lead, rest = t.shape[:2], t.shape[2:]
        n = int(np.prod(rest))
        pad = -(-n // 8) * 8
        wide = torch.full(tuple(lead) + (pad + n + pad,), float("nan"), dtype=td)
        wide[..., pad:pad + n] = t.reshape(*lead, n)
        return wide.cuda()[..., pad:pad + n].unflatten(-1, tuple(rest))
    return t.cuda()


def _host(t, bfirst=False):
    x = t.double().cpu().numpy()
    return np.swapaxes(x, 0, 1) if bfirst else x


def _close(got, want, tol, what):
    assert np.all(np.isfinite(got)), what
    n = np.linalg.norm(want)
    d = np.linalg.norm(got - want)
    assert d <= tol * n if n else d == 0, f"{what}: {d / n if n else d:.2e} > {tol:.1e}"


def _run(inp, dtype, bfirst=False, packed=False, lens=None, state=True, stream=None):
    import bwd_persistent_cta_gb300 as R
    torch = _torch()
    T, B, Hk, Dk = inp["q"].shape
    Hv, Dv = inp["v"].shape[2:]
    op = R.DeltaRule(B, T, Hk, Hv, Dk, Dv, dtype=dtype, batch_first=bfirst)
    if lens is not None:
        op.set_seq_lengths(list(lens))
    x = [_dev(inp[n], dtype, bfirst, packed) for n in ("q", "k", "v", "g", "beta")]
    s0 = torch.from_numpy(inp["s0"]).cuda() if state else None
    dsT = torch.from_numpy(inp["dsT"]).cuda() if state else None
    do = _dev(inp["do"], dtype, bfirst)
    torch.cuda.synchronize()
    o, sT = op.forward(*x, s0=s0, stream=stream)
    grads = op.backward(do, *x, s0=s0, dsT=dsT, stream=stream)
    torch.cuda.synchronize()
    assert op.launches() >= 3
    out = {"o": _host(o, bfirst), "sT": _host(sT), "ds0": _host(grads[5])}
    for n, t in zip(("dq", "dk", "dv", "dg", "dbeta"), grads):
        out[n] = _host(t, bfirst)
    o2, s2 = op.forward(*x, s0=s0, train=False)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(sT, s2), "inference and training forward differ"
    return out


def _want(inp, lens=None, state=True):
    a = [np.nan_to_num(inp[n]) if n not in ("g",) else inp[n] for n in ("q", "k", "v", "g", "beta")]
    s0, dsT = (inp["s0"], inp["dsT"]) if state else (None, None)
    o, sT, kept = O.delta_forward(*a, s0, lens)
    dq, dk, dv, dg, db, ds0 = O.delta_backward(np.nan_to_num(inp["do"]), *a, sT, kept, dsT, lens)
    return dict(o=o, sT=sT, dq=dq, dk=dk, dv=dv, dg=dg, dbeta=db, ds0=ds0)


def _compare(got, want, dtype):
    for n, w in want.items():
        _close(got[n], w, (STATE_TOL if n in ("sT", "ds0") else TOL)[dtype], n)


SHAPES = [
    # T, B, Hk, Hv, Dk, Dv
    (1, 1, 1, 1, 64, 64),
    (1, 3, 2, 4, 128, 128),
    (2, 2, 1, 1, 64, 128),
    (15, 1, 1, 2, 128, 64),
    (16, 2, 1, 1, 128, 128),
    (17, 1, 2, 2, 64, 64),
    (31, 2, 1, 1, 64, 64),
    (33, 1, 1, 3, 64, 64),
    (63, 1, 1, 1, 128, 128),
    (64, 2, 1, 2, 128, 128),
    (65, 1, 3, 3, 128, 128),
    (127, 1, 1, 1, 64, 128),
    (200, 2, 2, 4, 128, 128),
    (321, 1, 1, 1, 128, 256),
    # widths that no tile divides
    (40, 2, 1, 2, 8, 8),
    (70, 1, 1, 1, 24, 40),
    (37, 1, 2, 2, 96, 192),
    (50, 1, 1, 1, 256, 256),
    (66, 1, 1, 1, 128, 72),
    (35, 1, 1, 2, 200, 128),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_shapes(shape, dtype):
    T, B, Hk, Hv, Dk, Dv = shape
    inp = _inputs(*shape, dtype, 11 + T)
    _compare(_run(inp, dtype), _want(inp), dtype)


@pytest.mark.parametrize("shape", [(100, 1, 1, 2, 64, 96), (90, 1, 1, 1, 128, 32), (70, 2, 1, 1, 128, 160),
                                   (66, 1, 2, 2, 64, 256)], ids=str)
def test_value_widths_on_tensor_cores(shape):
    inp = _inputs(*shape, "bf16", 15 + shape[5])
    _compare(_run(inp, "bf16"), _want(inp), "bf16")


@pytest.mark.parametrize("shape", [(130, 2, 25, 50, 64, 128), (130, 1, 25, 50, 128, 128), (130, 1, 20, 80, 64, 64),
                                   (70, 2, 80, 80, 128, 128)], ids=str)
def test_many_heads(shape):
    """Enough heads that one CTA takes four and eight slices of a head's value columns, and more than one turn."""
    T, B = shape[:2]
    inp = _inputs(*shape, "bf16", 17)
    lens = [T, T - 37][:B]
    _compare(_run(inp, "bf16", bfirst=True, lens=lens), _want(inp, lens), "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bfirst", [False, True])
def test_packed_rows_and_masked_garbage(dtype, bfirst):
    """Slices of packed projections, unequal lengths (0, 1, a chunk's edge and around it, all), NaN and infinity in what
    the masks hide."""
    lens = [0, 1, 64, 63, 65, 130, 128, 32]
    T, B = 130, len(lens)
    inp = _inputs(T, B, 2, 4, 64, 64, dtype, 21)
    for b, n in enumerate(lens):
        for name, bad in (("q", np.nan), ("k", np.inf), ("v", -np.inf), ("g", np.nan), ("beta", np.nan), ("do", np.inf)):
            inp[name][n:, b] = bad
    clean = {n: np.where(np.isfinite(x), x, 0.0) for n, x in inp.items()}
    got = _run(inp, dtype, bfirst, packed=True, lens=lens)
    _compare(got, _want(clean, lens), dtype)
    for b, n in enumerate(lens):
        for name in ("o", "dq", "dk", "dv", "dg", "dbeta"):
            assert np.all(got[name][n:, b] == 0.0), (name, b)
    np.testing.assert_array_equal(got["sT"][0], inp["s0"][0].astype(np.float64))
    np.testing.assert_array_equal(got["ds0"][0], inp["dsT"][0].astype(np.float64))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_state_given(dtype):
    inp = _inputs(100, 2, 1, 2, 128, 128, dtype, 31)
    _compare(_run(inp, dtype, state=False), _want(inp, state=False), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_resets_strong_decay_and_no_writes(dtype):
    """g = -inf (a document boundary) at the edges of chunks and inside, decays that underflow, the dtype's lowest value,
    beta of zero and one."""
    T = 150
    inp = _inputs(T, 2, 1, 2, 64, 64, dtype, 41)
    for t in (0, 5, 31, 32, 64, 100):
        inp["g"][t, 0] = -np.inf
    inp["g"][70:90, 1] = -40.0
    inp["g"][110, 1] = -3.3895313892515355e38
    inp["beta"][10:40, :, 0] = 0.0
    inp["beta"][50:60] = 1.0
    with np.errstate(invalid="ignore"):
        want = _want(inp)
    _compare(_run(inp, dtype), want, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["q", "k", "v", "beta"])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_bad_values_show(dtype, name, bad):
    """A NaN or an infinity in a valid token reaches that token's output or its state, and nothing turns into a wrong
    finite number: what is finite is right, and earlier chunks and other sequences are untouched."""
    import bwd_persistent_cta_gb300 as R
    torch = _torch()
    T, B, H, D = 150, 2, 1, 64
    inp = _inputs(T, B, H, H, D, D, dtype, 45)
    a = [inp[n] for n in ("q", "k", "v", "g", "beta")]
    wo, ws, _ = O.delta_forward(*a, inp["s0"])
    x = {n: inp[n].copy() for n in ("q", "k", "v", "g", "beta")}
    x[name][70, 0] = bad
    op = R.DeltaRule(B, T, H, H, D, D, dtype=dtype)
    o, sT = op.forward(*(_dev(x[n], dtype) for n in ("q", "k", "v", "g", "beta")), s0=torch.from_numpy(inp["s0"]).cuda(),
                       train=False)
    o, sT = _host(o), _host(sT)
    _close(o[:64, 0], wo[:64, 0], TOL[dtype], "earlier chunk")
    _close(o[:, 1], wo[:, 1], TOL[dtype], "other sequence")
    _close(sT[1], ws[1], STATE_TOL[dtype], "other state")
    assert not np.all(np.isfinite(o[70, 0]))
    fine = np.isfinite(o[64:70, 0])
    d = np.abs(o[64:70, 0] - wo[64:70, 0])[fine]
    assert np.all(d <= 40 * TOL[dtype] * np.abs(wo).max())
    if name != "q":
        assert not np.all(np.isfinite(o[71:, 0])) and not np.all(np.isfinite(sT[0]))
        assert not np.any(np.isfinite(o[128:, 0]).all(-1))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_keys(dtype):
    """One key repeated with full write strength, the worst case for the inverse inside a chunk: the state holds the last
    value exactly."""
    inp = _inputs(96, 1, 1, 1, 64, 64, dtype, 51, gate=1e-3)
    inp["k"][:] = 0.0
    inp["k"][..., 3] = 1.0
    inp["beta"][:] = 1.0
    _compare(_run(inp, dtype), _want(inp), dtype)


def test_gradient_against_differences():
    """The fp32 gradients along random directions against central differences of the fp64 forward (truncation 1e-8
    of the value, so the bound is the gradients' own)."""
    shape = (70, 1, 1, 2, 64, 64)
    inp = _inputs(*shape, "f32", 61)
    got = _run(inp, "f32")
    rng = np.random.default_rng(62)
    names = ("q", "k", "v", "g", "beta", "s0")
    for i, n in enumerate(names):
        d = rng.normal(size=inp[n].shape)
        d /= np.linalg.norm(d)

        def loss(h):
            a = [inp[m] + (h * d if m == n else 0.0) for m in names]
            o, s, _ = O.delta_forward(*a)
            return (o * inp["do"]).sum() + (s * inp["dsT"]).sum()

        want = (loss(1e-4) - loss(-1e-4)) / 2e-4
        grad = got["d" + n]
        assert abs((grad * d).sum() - want) <= 1e-5 * np.linalg.norm(grad) + 1e-7, n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_repeats_are_bit_identical(dtype):
    inp = _inputs(333, 3, 2, 4, 128, 128, dtype, 71)
    a, b = _run(inp, dtype), _run(inp, dtype)
    for n in a:
        np.testing.assert_array_equal(a[n], b[n], err_msg=n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_another_stream(dtype):
    torch = _torch()
    inp = _inputs(90, 2, 1, 2, 128, 128, dtype, 81)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = _run(inp, dtype, stream=s)
    _compare(got, _want(inp), dtype)


def test_long_sequence():
    """Many chunks; the reference's cost bounds the length."""
    inp = _inputs(2500, 1, 1, 2, 128, 128, "bf16", 91)
    _compare(_run(inp, "bf16"), _want(inp), "bf16")


# --- the serving step ---------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,B,Hk,Hv,Dk,Dv", [(1, 1, 1, 1, 64, 64), (1, 5, 2, 4, 128, 128), (3, 4, 1, 3, 128, 64),
                                             (1, 3, 2, 2, 24, 40), (2, 2, 1, 1, 256, 256), (5, 2, 1, 2, 64, 128)])
def test_step(T, B, Hk, Hv, Dk, Dv, dtype):
    """Slots in any order in a larger pool, an unused slot untouched, slots outside the pool skipped."""
    import bwd_persistent_cta_gb300 as R
    torch = _torch()
    inp = _inputs(T, B, Hk, Hv, Dk, Dv, dtype, 100 + T + B)
    pool = B + 3
    rng = np.random.default_rng(7)
    state = rng.normal(size=(pool, Hv, Dv, Dk)).astype(np.float32)
    slots = rng.permutation(pool)[:B].astype(np.int32)
    skipped = {}
    if B > 2:
        skipped = {0: -1, 2: pool}
    for b, s in skipped.items():
        slots[b] = s
    x = [_dev(inp[n], dtype, packed=True) for n in ("q", "k", "v", "g", "beta")]
    op = R.DeltaRule(B, T, Hk, Hv, Dk, Dv, dtype=dtype)
    st = torch.from_numpy(state.copy()).cuda()
    o = _host(op.step(*x, st, slots=torch.from_numpy(slots).cuda()))
    st = st.cpu().numpy()
    a = [inp[n] for n in ("q", "k", "v", "g", "beta")]
    s0 = np.stack([state[s] if 0 <= s < pool else np.zeros_like(state[0]) for s in slots])
    wo, ws, _ = O.delta_forward(*a, s0)
    want = state.astype(np.float64)
    for b, s in enumerate(slots):
        if b in skipped:
            assert np.all(o[:, b] == 0.0)
            wo[:, b] = 0.0
        else:
            want[s] = ws[b]
    _close(o, wo, TOL[dtype], "o")
    _close(st.astype(np.float64), want, TOL["f32"], "state")
    untouched = sorted(set(range(pool)) - {int(s) for s in slots})
    np.testing.assert_array_equal(st[untouched], state[untouched])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,B,Hk,Hv,Dk,Dv", [(1, 70, 2, 8, 128, 128), (2, 61, 4, 8, 64, 128), (1, 130, 3, 3, 96, 72),
                                             (2, 80, 8, 8, 24, 40), (3, 61, 4, 8, 64, 128), (1, 40, 8, 8, 256, 128)])
def test_step_many(T, B, Hk, Hv, Dk, Dv, dtype):
    """Enough states for every CTA to walk several: odd widths, a different number of tokens (none included) for each
    sequence, slots outside the pool, garbage behind the masks."""
    import bwd_persistent_cta_gb300 as R
    torch = _torch()
    inp = _inputs(T, B, Hk, Hv, Dk, Dv, dtype, 300 + B)
    lens = [(b * 5 + 1) % (T + 1) if T > 1 else 1 for b in range(B)]
    for b, n in enumerate(lens):
        for name in ("q", "k", "v", "g", "beta"):
            inp[name][n:, b] = np.nan
    pool = B + 9
    rng = np.random.default_rng(8)
    state = rng.normal(size=(pool, Hv, Dv, Dk)).astype(np.float32)
    slots = rng.permutation(pool)[:B].astype(np.int32)
    skipped = {3: -1, 17: pool, 30: 2 ** 31 - 1}
    for b, s in skipped.items():
        slots[b] = s
    op = R.DeltaRule(B, T, Hk, Hv, Dk, Dv, dtype=dtype, batch_first=True)
    op.set_seq_lengths(lens)
    st = torch.from_numpy(state.copy()).cuda()
    x = [_dev(inp[n], dtype, bfirst=True, packed=True) for n in ("q", "k", "v", "g", "beta")]
    sl = torch.from_numpy(slots).cuda()
    o = _host(op.step(*x, st, slots=sl), True)
    op.sync()
    st = st.cpu().numpy()
    a = [np.nan_to_num(inp[n]) for n in ("q", "k", "v", "g", "beta")]
    ok = [b for b in range(B) if b not in skipped]
    s0 = np.stack([state[s] if 0 <= s < pool else np.zeros_like(state[0]) for s in slots])
    wo, ws, _ = O.delta_forward(*a, s0, lens)
    want = state.astype(np.float64)
    for b in ok:
        want[slots[b]] = ws[b]
    for b in skipped:
        wo[:, b] = 0.0
    _close(o, wo, TOL[dtype], "o")
    _close(st.astype(np.float64), want, TOL["f32"], "state")
    for b in range(B):
        assert np.all(o[lens[b]:, b] == 0.0)
        if lens[b] == 0 and b not in skipped:
            np.testing.assert_array_equal(st[slots[b]], state[slots[b]])
    for b in skipped:
        assert np.all(o[:, b] == 0.0)


def test_step_lengths():
    """A different number of accepted tokens for each sequence, none of them included."""
    import bwd_persistent_cta_gb300 as R
    torch = _torch()
    lens = [0, 1, 4, 3, 2]
    T, B = 4, len(lens)
    inp = _inputs(T, B, 1, 2, 128, 128, "bf16", 111)
    for b, n in enumerate(lens):
        for name in ("q", "k", "v", "g", "beta"):
            inp[name][n:, b] = np.nan
    op = R.DeltaRule(B, T, 1, 2, 128, 128)
    op.set_seq_lengths(lens)
    st = torch.from_numpy(inp["s0"]).cuda().clone()
    o = _host(op.step(*(_dev(inp[n], "bf16") for n in ("q", "k", "v", "g", "beta")), st))
    a = [np.nan_to_num(inp[n]) for n in ("q", "k", "v", "g", "beta")]
    wo, ws, _ = O.delta_forward(*a, inp["s0"], lens)
    _close(o, wo, TOL["bf16"], "o")
    _close(st.double().cpu().numpy(), ws, TOL["f32"], "state")
    np.testing.assert_array_equal(st[0].cpu().numpy(), inp["s0"][0])


def test_prefill_then_steps_is_one_sequence():
    import bwd_persistent_cta_gb300 as R
    torch = _torch()
    T, n = 75, 70
    inp = _inputs(T, 2, 1, 2, 128, 128, "bf16", 121)
    x = [_dev(inp[m], "bf16") for m in ("q", "k", "v", "g", "beta")]
    pre = R.DeltaRule(2, n, 1, 2, 128, 128)
    one = R.DeltaRule(2, 1, 1, 2, 128, 128)
    o, st = pre.forward(*(t[:n].contiguous() for t in x), train=False)
    outs = [o] + [one.step(*(t[i:i + 1].contiguous() for t in x), st) for i in range(n, T)]
    a = [inp[m] for m in ("q", "k", "v", "g", "beta")]
    wo, ws, _ = O.delta_forward(*a)
    _close(_host(torch.cat(outs)), wo, TOL["bf16"], "o")
    _close(st.double().cpu().numpy(), ws, STATE_TOL["bf16"], "state")


def test_step_offsets_past_32_bits():
    """A pool of more than 2^32 bytes and 2^31 elements, its last slot used."""
    import bwd_persistent_cta_gb300 as R
    torch = _torch()
    Hv = D = 128
    slots = (2 ** 31) // (Hv * D * D) + 8            # 2 MB x 4 a slot
    inp = _inputs(1, 1, Hv, Hv, D, D, "bf16", 131)
    st = torch.empty(slots, Hv, D, D, dtype=torch.float32, device="cuda")
    assert st.numel() > 2 ** 31
    st[-1] = torch.from_numpy(inp["s0"][0]).cuda()
    op = R.DeltaRule(1, 1, Hv, Hv, D, D)
    x = [_dev(inp[n], "bf16") for n in ("q", "k", "v", "g", "beta")]
    o = _host(op.step(*x, st, slots=torch.tensor([slots - 1], dtype=torch.int32, device="cuda")))
    wo, ws, _ = O.delta_forward(*(inp[n] for n in ("q", "k", "v", "g", "beta")), inp["s0"])
    _close(o, wo, TOL["bf16"], "o")
    _close(st[-1:].double().cpu().numpy(), ws, TOL["f32"], "state")


# --- refusals -----------------------------------------------------------------
def test_refusals():
    import bwd_persistent_cta_gb300 as R
    torch = _torch()
    op = R.DeltaRule(2, 3, 1, 2, 64, 64)
    L, bad = R.lib(), R.RNN_BAD_PARAM
    bf = torch.bfloat16
    q = torch.zeros(3, 2, 1, 64, dtype=bf, device="cuda")
    v = torch.zeros(3, 2, 2, 64, dtype=bf, device="cuda")
    g = torch.zeros(3, 2, 2, dtype=bf, device="cuda")
    st = torch.zeros(2, 2, 64, 64, device="cuda")
    P = lambda t: t.data_ptr()  # noqa: E731
    good = dict(q=P(q), k=P(q), v=P(v), g=P(g), beta=P(g))
    buf = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")

    def fwd(o=P(v), s0=None, sT=None, ws=P(buf), rs=None, **kw):
        return R.rnn_delta_forward(op.handle, R.rnn_delta_in_t(**{**good, **kw}), s0, o, sT, ws, rs)

    assert fwd() == R.RNN_OK
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(g=None), dict(beta=None), dict(q=P(q) + 2),
               dict(v=P(v) + 8), dict(g=P(g) + 1), dict(q_row=56), dict(q_row=68), dict(v_row=64), dict(g_row=1),
               dict(beta_row=-2), dict(o=None), dict(o=P(v) + 2), dict(s0=P(st) + 4), dict(sT=P(st) + 8)):
        assert fwd(**kw) == bad, kw
    assert fwd(rs=P(buf) + 4) == R.RNN_BAD_WORKSPACE
    x = R.rnn_delta_in_t(**good)
    grads = [P(q), P(q), P(v), P(g), P(g)]
    args = [P(v), None] + grads + [None, P(buf), P(buf)]
    for i in (0, 2, 3, 4, 5, 6):
        assert R.rnn_delta_backward(op.handle, x, *(args[:i] + [None] + args[i + 1:])) == bad, i
    for i in (8, 9):
        assert R.rnn_delta_backward(op.handle, x, *(args[:i] + [None] + args[i + 1:])) == R.RNN_BAD_WORKSPACE, i
    for a in ((None, 2, None, P(v)), (P(st), -1, None, P(v)), (P(st), 2, None, None), (P(st) + 4, 2, None, P(v)),
              (P(st), 2, P(buf) + 2, P(v))):
        assert R.rnn_delta_step(op.handle, x, *a) == bad, a
    assert R.rnn_delta_set_seq_lengths(op.handle, [4, 0]) == bad
    assert R.rnn_delta_set_seq_lengths(op.handle, [-1, 0]) == bad
    with pytest.raises(ValueError):
        op.forward(q.cpu(), q, v, g, g)
    with pytest.raises(ValueError):
        op.backward(v, q, q, v, g, g)                # no training forward yet
    torch.cuda.synchronize()
