"""The gated delta rule at edges of its range."""
import numpy as np
import pytest

from tests.test_delta_gpu import TOL, _close, _dev, _host, _inputs, _run, _want

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
