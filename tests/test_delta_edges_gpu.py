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
