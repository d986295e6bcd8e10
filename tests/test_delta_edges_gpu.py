"""The gated delta rule at edges of its range."""
import numpy as np
import pytest

from oracle import lm_oracle as O

from tests.test_delta_gpu import TOL, _close, _compare, _dev, _host, _inputs, _run, _want

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "g", "beta")
GRADS = ("dq", "dk", "dv", "dg", "dbeta")


@pytest.mark.parametrize("every", [2, 3, 4])
def test_fp32_gradients_between_resets(every):
    """A reset every few tokens, each token's gradient by itself, to the fp32 tolerance of whole tensors: a token's
    weight towards another is the decay between them, whatever lies before both."""
    T = 70
    inp = _inputs(T, 1, 1, 2, 64, 64, "f32", 501)
    inp["g"][::every] = -np.inf
    with np.errstate(invalid="ignore"):
        want = _want(inp)
    got = _run(inp, "f32")
    for n in ("dq", "dk", "dv", "dbeta"):
        for t in range(T):
            _close(got[n][t], want[n][t], TOL["f32"], f"{n} of token {t}")
    _close(got["dg"], want["dg"], TOL["f32"], "dg")


def test_bf16_gradients_do_not_depend_on_earlier_resets():
    """A document that starts inside a chunk gets the same gradients whether one boundary or forty lie before it in the
    chunk.  Both runs do the same arithmetic on the document, so an output differs only where an inner difference of a
    few 2^-23 of its size moves a rounding to bf16 (spacing 2^-8): below one in 2000.  A cumulative decay of 4500 held in
    24 bits would be off by 2^-12, and move one in 30."""
    T, at, H = 64, 40, 16
    inp = _inputs(T, 1, H, H, 128, 128, "bf16", 502)
    inp["g"][at] = -np.inf
    plain = _run(inp, "bf16")
    inp["g"][:at] = -np.inf
    many = _run(inp, "bf16")
    for n in ("o",) + GRADS:
        a, b = plain[n][at:], many[n][at:]
        assert np.mean(a != b) <= 1 / 500, (n, np.mean(a != b))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", NAMES + ("do",))
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_masked_tokens_stay_zero_beside_a_bad_value(dtype, name, bad):
    """A NaN or an infinity in a valid token shows, but not in the masked tokens of its chunk."""
    if name == "g" and bad == np.inf:
        bad = 1e30                                 # an infinite growth
    T, lens = 140, [71, 140, 0, 30]
    inp = _inputs(T, 4, 2, 4, 64, 64, dtype, 503)
    inp[name][70, 0] = bad
    inp[name][20, 3] = bad
    import bwd_persistent_cta_gb300 as R
    import torch
    op = R.DeltaRule(4, T, 2, 4, 64, 64, dtype=dtype)
    op.set_seq_lengths(lens)
    x = [_dev(inp[n], dtype) for n in NAMES]
    s0 = torch.from_numpy(inp["s0"]).cuda()
    o, sT = op.forward(*x, s0=s0)
    grads = op.backward(_dev(inp["do"], dtype), *x)
    out = dict(zip(GRADS, (_host(t) for t in grads)), o=_host(o))
    for n, t in out.items():
        for b, length in enumerate(lens):
            assert np.all(t[length:, b] == 0.0), (n, b)
    assert not all(np.all(np.isfinite(t[:71, 0])) for t in out.values())
    if name != "do":
        inp[name][70, 0] = inp[name][20, 3] = 0.5
        _close(out["o"][:, 1:3], _want(inp, lens)["o"][:, 1:3], TOL[dtype], "other sequences")


@pytest.mark.parametrize("H,D", [(70, 128), (160, 128), (160, 64)])
def test_masked_tokens_stay_zero_with_many_heads(H, D):
    """The same where a CTA takes four and eight slices of a head's value columns."""
    import bwd_persistent_cta_gb300 as R
    T, lens = 75, [70, 3]
    inp = _inputs(T, 2, H, H, D, D, "bf16", 506)
    inp["k"][66, 0] = inp["v"][1, 1] = np.nan
    op = R.DeltaRule(2, T, H, H, D, D)
    op.set_seq_lengths(lens)
    x = [_dev(inp[n], "bf16") for n in NAMES]
    o, _ = op.forward(*x)
    grads = op.backward(_dev(inp["do"], "bf16"), *x)
    for n, t in zip(("o",) + GRADS, (o,) + grads):
        t = _host(t)
        assert not np.all(np.isfinite(t)), n
        for b, length in enumerate(lens):
            assert np.all(t[length:, b] == 0.0), (n, b)


@pytest.mark.parametrize("seed", [1, 2, 3])
@pytest.mark.parametrize("T,Dk,Dv", [(513, 64, 128), (700, 128, 64)])
def test_fp32_error_does_not_grow_with_the_sequence(T, Dk, Dv, seed):
    """Memories of a hundred to a thousand tokens.  16 * 2^-24 = 9.5e-7 for every tensor: a value passes sums of at most
    256 products in trees or chains of 32 (below 6 * 2^-24 with random signs) and a dozen single roundings; no term counts
    the tokens of the sequence, which would be another 2^-24 sqrt(T) = 23 * 2^-24 and more."""
    tol = 16 * 2.0 ** -24
    inp = _inputs(T, 1, 1, 2, Dk, Dv, "f32", 520 + seed, gate=0.05)
    got, want = _run(inp, "f32"), _want(inp)
    for n, w in want.items():
        _close(got[n], w, tol, n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta"])
def test_finite_outputs_beside_a_bad_value_are_right(dtype, name):
    """What stays finite in the sequence that holds a NaN is what it would be without it."""
    import bwd_persistent_cta_gb300 as R
    import torch
    T, B, H, D = 150, 1, 1, 64
    inp = _inputs(T, B, H, H, D, D, dtype, 504)
    a = [inp[n] for n in NAMES]
    wo, _, _ = O.delta_forward(*a, inp["s0"])
    x = {n: inp[n].copy() for n in NAMES}
    x[name][70, 0] = np.nan
    op = R.DeltaRule(B, T, H, H, D, D, dtype=dtype)
    o, sT = op.forward(*(_dev(x[n], dtype) for n in NAMES), s0=torch.from_numpy(inp["s0"]).cuda(), train=False)
    o = _host(o)
    _close(o[:64], wo[:64], TOL[dtype], "earlier chunk")
    assert not np.all(np.isfinite(o[70]))
    d = np.abs(o - wo)[np.isfinite(o)]
    assert np.all(d <= 40 * TOL[dtype] * np.abs(wo).max())
    if name != "q":
        assert not np.any(np.isfinite(o[128:]).all(-1)) and not np.all(np.isfinite(_host(sT)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,B,Hk,Hv,Dk,Dv", [(8, 5, 1, 2, 64, 64), (17, 6, 2, 4, 128, 128), (33, 5, 2, 2, 128, 64),
                                             (9, 4, 1, 1, 24, 40), (20, 3, 1, 1, 256, 72)])
def test_step_of_many_tokens(T, B, Hk, Hv, Dk, Dv, dtype):
    """Slots in any order, slots outside the pool, sequences of every length down to none, garbage behind the masks."""
    import bwd_persistent_cta_gb300 as R
    import torch
    inp = _inputs(T, B, Hk, Hv, Dk, Dv, dtype, 505 + T)
    lens = [T, 0, T - 1, 1, T // 2, 8][:B]
    for b, n in enumerate(lens):
        for name in NAMES:
            inp[name][n:, b] = np.nan
    pool = B + 4
    rng = np.random.default_rng(9)
    state = rng.normal(size=(pool, Hv, Dv, Dk)).astype(np.float32)
    slots = rng.permutation(pool)[:B].astype(np.int32)
    skipped = {2: -1} if B < 5 else {2: -1, 4: pool}
    for b, s in skipped.items():
        slots[b] = s
    op = R.DeltaRule(B, T, Hk, Hv, Dk, Dv, dtype=dtype, batch_first=True)
    op.set_seq_lengths(lens)
    st = torch.from_numpy(state.copy()).cuda()
    x = [_dev(inp[n], dtype, bfirst=True, packed=True) for n in NAMES]
    o = _host(op.step(*x, st, slots=torch.from_numpy(slots).cuda()), True)
    st = st.cpu().numpy()
    a = [np.nan_to_num(inp[n]) for n in NAMES]
    s0 = np.stack([state[s] if 0 <= s < pool else np.zeros_like(state[0]) for s in slots])
    wo, ws, _ = O.delta_forward(*a, s0, lens)
    want = state.astype(np.float64)
    for b in range(B):
        if b in skipped:
            wo[:, b] = 0.0
        else:
            want[slots[b]] = ws[b]
        assert np.all(o[lens[b]:, b] == 0.0)
    _close(o, wo, TOL[dtype], "o")
    _close(st.astype(np.float64), want, TOL["f32"], "state")
    same = sorted(set(range(pool)) - {int(slots[b]) for b in range(B) if b not in skipped and lens[b]})
    np.testing.assert_array_equal(st[same], state[same])


@pytest.mark.parametrize("T,B,Hk,Hv,Dk,Dv", [(1500, 2, 1, 2, 128, 128), (1000, 1, 2, 4, 64, 96), (300, 1, 80, 80, 128, 128)])
def test_bf16_states_hold_22_bits(T, B, Hk, Hv, Dk, Dv):
    """States behind bf16 sequences.  What reaches a state is held as pairs of fp16, 22 bits below the largest of a tile:
    four products on a value's way, each with up to three terms of 2^-23 of it, is 12 * 2^-23 = 1.4e-6."""
    inp = _inputs(T, B, Hk, Hv, Dk, Dv, "bf16", 530, gate=0.2)
    got, want = _run(inp, "bf16"), _want(inp)
    for n in ("sT", "ds0"):
        _close(got[n], want[n], 12 * 2.0 ** -23, n)


@pytest.mark.parametrize("shape", [(75, 8, 8, 16, 64, 64), (70, 4, 16, 16, 128, 128), (40, 16, 16, 16, 24, 40),
                                   (40, 2, 16, 16, 256, 256)], ids=str)
def test_fp32_with_many_rows(shape):
    """Enough rows of state that a warp takes eight, with lengths."""
    T, B = shape[:2]
    inp = _inputs(*shape, "f32", 540)
    lens = [T - (b * T) // B for b in range(B)]
    _compare(_run(inp, "f32", lens=lens, packed=True), _want(inp, lens), "f32")
