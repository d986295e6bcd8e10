"""SelectiveScan, CausalConv and GradClip on streams, in graphs and in the order of their
calls.  A device-side delay holds one stream back, so that what is not ordered happens
in the wrong order."""
import numpy as np
import pytest

from oracle import ssm_oracle as O

from tests.test_conv_gpu import _inputs as conv_inputs
from tests.test_lm_streams_gpu import _busy_block, _delay
from tests.test_scan_gpu import OUT_TOL, STATE_TOL, _close, _inputs, _np

pytestmark = pytest.mark.gpu

ARGS = ("x", "dt", "A", "Bm", "Cm")
MORE = ("z", "D", "dt_bias")


def _scan(t):
    dev = {n: v.cuda() for n, v in t.items()}
    return [dev[n] for n in ARGS], {n: dev[n] for n in MORE}, dev


def _want(t, lengths=None, h0=None):
    host = {n: _np(v) for n, v in t.items()}
    return O.scan_forward(*(host[n] for n in ARGS), *(host[n] for n in MORE), h0, lengths)


@pytest.mark.parametrize("T", [40, 300])
def test_lengths_change_behind_a_queued_scan(T):
    import torch
    import bwd_persistent_cta_gb300 as R
    first, second = [T, 5], [9, T - 1]
    t = _inputs(T, 2, 24, 16, 1, "bf16", 21)
    args, kw, _ = _scan(t)
    op = R.SelectiveScan(2, T, 24, 16)
    op.forward(*args, **kw, train=False)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        op.set_seq_lengths(first)
        _delay()
        got = [op.forward(*args, **kw, train=False)]
        op.set_seq_lengths(second)
        got.append(op.forward(*args, **kw, train=False))
    torch.cuda.synchronize()
    for lens, (y, hT) in zip((first, second), got):
        wy, wh, _ = _want(t, lens)
        _close(y, wy, OUT_TOL["bf16"], f"y of {lens}")
        _close(hT, wh, STATE_TOL["bf16"], f"state of {lens}")


def test_lengths_change_behind_queued_steps_and_convolutions():
    import torch
    import bwd_persistent_cta_gb300 as R
    t = conv_inputs(6, 3, 40, 4, "bf16", 22)
    dev = {n: v.cuda() for n, v in t.items()}
    op = R.CausalConv(3, 6, 40, 4)
    st = t["s0"].cuda()
    s = torch.cuda.Stream()
    op.forward(dev["x"], dev["w"])
    op.step(dev["x"], dev["w"], st.clone())
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        op.set_seq_lengths([6, 0, 2])
        _delay()
        y, sT = op.forward(dev["x"], dev["w"], s0=dev["s0"])
        op.step(dev["x"], dev["w"], st)
        op.set_seq_lengths([1, 6, 3])
        op.step(dev["x"], dev["w"], st)
    torch.cuda.synchronize()
    _, w1, _ = O.conv_forward(_np(t["x"]), _np(t["w"]), None, _np(t["s0"]), [6, 0, 2])
    assert np.array_equal(_np(sT.cpu()), w1)
    _, w2, _ = O.conv_forward(_np(t["x"]), _np(t["w"]), None, w1, [1, 6, 3])
    assert np.array_equal(_np(st.cpu()), w2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_later_call_on_another_stream_keeps_the_reserve(dtype):
    import torch
    import bwd_persistent_cta_gb300 as R
    T, B, D, N = 150, 2, 40, 16
    one, two = (_inputs(T, B, D, N, 1, dtype, s) for s in (23, 24))
    (a1, k1, d1), (a2, k2, _) = _scan(one), _scan(two)
    op = R.SelectiveScan(B, T, D, N, dtype=dtype)
    op.forward(*a1, **k1)
    want = op.backward(d1["dy"], *a1, **k1)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s1):
        op.forward(*a1, **k1)
        _delay()
        got = op.backward(d1["dy"], *a1, **k1)
    with torch.cuda.stream(s2):
        op.forward(*a2, **k2)
    torch.cuda.synchronize()
    for n in want:
        assert torch.equal(got[n], want[n]), n


def test_calls_that_share_scratch_run_in_order():
    """Segments' ends, the convolution's partial sums and the norm's lie in the handle's scratch."""
    import torch
    import bwd_persistent_cta_gb300 as R
    t = _inputs(400, 1, 24, 16, 1, "bf16", 25)
    args, kw, _ = _scan(t)
    scan = R.SelectiveScan(1, 400, 24, 16)
    c = {n: v.cuda() for n, v in conv_inputs(50, 2, 40, 4, "bf16", 26).items()}
    conv = R.CausalConv(2, 50, 40, 4)
    g = [torch.randn(5000, device="cuda")]
    clip = R.GradClip([5000])
    for call in (lambda: scan.forward(*args, **kw, train=False), lambda: conv.backward(c["dy"], c["x"], c["w"]),
                 lambda: clip.norm(g)):
        call()
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        first, second = torch.cuda.Event(), torch.cuda.Event()
        with torch.cuda.stream(s1):
            _delay()
            call()
            first.record()
        with torch.cuda.stream(s2):
            call()
            second.record()
        second.synchronize()
        assert first.query()


def test_captured_training_and_clipping():
    """A training step, captured once and replayed on other values, is the eager one."""
    import torch
    import bwd_persistent_cta_gb300 as R
    T, B, D, N, W = 200, 2, 40, 16, 4
    t, t2 = (_inputs(T, B, D, N, 1, "bf16", s) for s in (27, 28))
    args, kw, dev = _scan(t)
    w = torch.randn(D, W, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    conv, scan = R.CausalConv(B, T, D, W), R.SelectiveScan(B, T, D, N)
    clip = R.GradClip([D * W, D * N, D], ["f32"] * 3)

    def step():
        xc, _ = conv.forward(dev["x"], w)
        ins = [xc] + args[1:]
        y, hT = scan.forward(*ins, **kw)
        d = scan.backward(dev["dy"], *ins, **kw)
        c = conv.backward(d["dx"], dev["x"], w)
        grads = [c["dw"], d["dA"], d["dD"]]
        norm = clip.clip(grads, 0.5)
        return [y, hT, c["dx"], d["ddt"], d["dB"], d["dC"], norm] + grads

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for src in (t2, t):
        for n in ("x", "dt", "z", "Bm", "Cm", "dy"):
            dev[n].copy_(src[n])
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_outputs_on_a_stream_that_is_not_current():
    """With ``stream=``, outputs do not take memory that the current stream has yet to read."""
    import torch
    import bwd_persistent_cta_gb300 as R
    s = torch.cuda.Stream()
    B, T, D, N = 4, 256, 2048, 16                 # 4 MB and more: blocks of their own
    t = {n: v.cuda() for n, v in _inputs(T, B, D, N, 1, "bf16", 29).items()}
    args = [t[n] for n in ARGS]
    scan, one, conv = R.SelectiveScan(B, T, D, N), R.SelectiveScan(B, 1, D, N), R.CausalConv(B, T, D, 4)
    w, st = torch.randn(D, 4, device="cuda").bfloat16(), torch.zeros(B, D, N, device="cuda")
    flat = t["x"].float().flatten()
    clip = R.GradClip([flat.numel()])
    cut = [a[:1].contiguous() if n != "A" else a for n, a in zip(ARGS, args)]
    calls = [(t["x"], lambda: scan.forward(*args, train=False, stream=s)),
             (t["x"], lambda: (scan.forward(*args, stream=s), scan.backward(t["dy"], *args, stream=s))),
             (t["x"], lambda: conv.forward(t["x"], w, stream=s)),
             (t["x"], lambda: conv.backward(t["dy"], t["x"], w, stream=s)),
             (cut[0], lambda: one.step(*cut, st, stream=s)),
             (flat[:1], lambda: clip.norm([flat], stream=s))]
    for like, call in calls:
        call()
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        kept = _busy_block(like)
        out = call()
        torch.cuda.synchronize()
        assert torch.all(kept == 3.0)
        del out


def test_gradients_dropped_while_another_stream_clips_them():
    import torch
    import bwd_persistent_cta_gb300 as R
    n = 1 << 22
    op = R.GradClip([n, n])
    g = [torch.full((n,), 2.0, device="cuda") for _ in range(2)]
    out = [torch.zeros(n, device="cuda") for _ in range(2)]
    op.clip(g, 1.0, out=out)
    want = [o.clone() for o in out]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        _delay()
    op.clip(g, 1.0, out=out, stream=s)
    del g
    others = [torch.zeros(n, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want)) and not any(o.any() for o in others)


def test_a_stream_of_another_device_is_refused():
    import torch
    import bwd_persistent_cta_gb300 as R

    class Other:
        device, cuda_stream = torch.device("cuda", 7), 0

    with pytest.raises(ValueError, match="stream"):
        R.GradClip([4]).clip([torch.zeros(4, device="cuda")], 1.0, stream=Other())
    with pytest.raises(ValueError, match="stream"):
        R.CausalConv(1, 1, 8).forward(torch.zeros(1, 1, 8, device="cuda").bfloat16(),
                                      torch.zeros(8, 4, device="cuda").bfloat16(), stream=Other())
