"""Sequences that run as several segments side by side, shown by the extra pass each
direction launches: groups, every width of state, unequal lengths, the state in place.
Inputs, reference and tolerances (for up to 600 tokens) are test_scan_gpu.py's."""
import pytest

from tests.test_scan_gpu import _inputs, run

pytestmark = pytest.mark.gpu

ARGS = ("x", "dt", "A", "Bm", "Cm")


def _in_segments(T, B, D, N, G, dtype):
    """Whether a handle of this shape has the extra passes: 1 + 1 launches forward, 3 + 1 backward."""
    import bwd_persistent_cta_gb300 as R
    t = {n: v.cuda() for n, v in _inputs(T, B, D, N, G, dtype, 1).items()}
    op = R.SelectiveScan(B, T, D, N, groups=G, dtype=dtype)
    args = [t[n] for n in ARGS]
    op.forward(*args)
    forward = op.launches()
    op.backward(t["dy"], *args)
    return forward == 2 and op.launches() - forward == 4


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,N,G", [(513, 48, 16, 2), (520, 72, 16, 3), (513, 528, 16, 2), (400, 48, 24, 2), (400, 72, 32, 3),
                                     (513, 32, 64, 2), (600, 96, 8, 4), (330, 24, 40, 1)])
def test_groups_and_widths(T, D, N, G, dtype):
    assert _in_segments(T, 2, D, N, G, dtype)
    run(T, 2, D, N, G, dtype=dtype, packed=True)
    run(T, 2, D, N, G, dtype=dtype, lengths=[T // 3 + 5, T - 1], bfirst=True, poison=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [16, 24])
def test_training_with_the_state_in_place(N, dtype):
    import torch
    import bwd_persistent_cta_gb300 as R
    T, B, D = 512, 2, 24
    assert _in_segments(T, B, D, N, 1, dtype)
    t = {n: v.cuda() for n, v in _inputs(T, B, D, N, 1, dtype, 12).items()}
    op = R.SelectiveScan(B, T, D, N, dtype=dtype)
    args, kw = [t[n] for n in ARGS], {n: t[n] for n in ("z", "D", "dt_bias")}
    y, hT = op.forward(*args, **kw, h0=t["h0"])
    want = op.backward(t["dy"], *args, **kw, dhT=t["dhT"])
    for _ in range(3):
        h = t["h0"].clone()
        y2, h2 = op.forward(*args, **kw, h0=h, hT=h)
        assert h2.data_ptr() == h.data_ptr() and torch.equal(y, y2) and torch.equal(hT, h2)
        got = op.backward(t["dy"], *args, **kw, dhT=t["dhT"])
        for n in want:
            assert torch.equal(got[n], want[n]), n
