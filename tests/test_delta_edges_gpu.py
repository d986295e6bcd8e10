"""The gated delta rule at edges of its range."""
import numpy as np
import pytest

from tests.test_delta_gpu import TOL, _close, _inputs, _run, _want

pytestmark = pytest.mark.gpu


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
    for n in ("o", "dq", "dk", "dv", "dg", "dbeta"):
        a, b = plain[n][at:], many[n][at:]
        assert np.mean(a != b) <= 1 / 500, (n, np.mean(a != b))
