"""Calls of DeltaRule and BlockNorm on streams.  A device-side delay holds one
stream back, so that what is not ordered happens in the wrong order."""
import numpy as np
import pytest

from oracle import lm_oracle as O

from tests.test_delta_gpu import STATE_TOL, TOL, _close, _dev, _host, _inputs

pytestmark = pytest.mark.gpu

NAMES = ("q", "k", "v", "g", "beta")
DELAY = 400_000_000            # cycles: about 0.2 s


def _delay():
    import torch
    torch.cuda._sleep(DELAY)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lengths_change_behind_a_queued_forward(dtype):
    import torch
    import bwd_persistent_cta_gb300 as R
    T, B, H, D = 130, 3, 2, 64
    first, second = [130, 20, 65], [3, 128, 0]
    inp = _inputs(T, B, H, H, D, D, dtype, 401)
    a = [inp[n] for n in NAMES]
    op = R.DeltaRule(B, T, H, H, D, D, dtype=dtype)
    s = torch.cuda.Stream()
    x = [_dev(t, dtype) for t in a]
    s0 = torch.from_numpy(inp["s0"]).cuda()
    op.forward(*x, s0=s0, train=False)           # a kernel's first launch may wait for the device
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        op.set_seq_lengths(first)
        _delay()
        got = [op.forward(*x, s0=s0, train=False)]
        op.set_seq_lengths(second)
        got.append(op.forward(*x, s0=s0, train=False))
    torch.cuda.synchronize()
    for lens, (o, sT) in zip((first, second), got):
        wo, ws, _ = O.delta_forward(*a, inp["s0"], lens)
        _close(_host(o), wo, TOL[dtype], f"o of lengths {lens}")
        _close(_host(sT), ws, STATE_TOL[dtype], f"state of lengths {lens}")


@pytest.mark.parametrize("T", [3, 12])
def test_lengths_change_behind_a_queued_step(T):
    import torch
    import bwd_persistent_cta_gb300 as R
    B, H, D = 3, 2, 64
    first, second = [T, 1, 2], [1, T, 0]
    inp = _inputs(T, B, H, H, D, D, "bf16", 402)
    a = [inp[n] for n in NAMES]
    op = R.DeltaRule(B, T, H, H, D, D)
    s = torch.cuda.Stream()
    x = [_dev(t, "bf16") for t in a]
    st = torch.from_numpy(inp["s0"]).cuda()
    op.step(*x, st.clone())
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        op.set_seq_lengths(first)
        _delay()
        o1 = op.step(*x, st)
        op.set_seq_lengths(second)
        o2 = op.step(*x, st)
    torch.cuda.synchronize()
    w1, ws, _ = O.delta_forward(*a, inp["s0"], first)
    w2, ws, _ = O.delta_forward(*a, ws, second)
    _close(_host(o1), w1, TOL["bf16"], "first")
    _close(_host(o2), w2, TOL["bf16"], "second")
    _close(_host(st), ws, TOL["f32"], "state")


def test_lengths_change_between_a_captured_graphs_replays():
    """A graph reads the lengths that are set when it runs; setting new ones waits for a replay in flight."""
    import torch
    import bwd_persistent_cta_gb300 as R
    T, B, H, D = 40, 2, 1, 64
    first, second = [40, 7], [12, 33]
    inp = _inputs(T, B, H, H, D, D, "bf16", 403)
    a = [inp[n] for n in NAMES]
    op = R.DeltaRule(B, T, H, H, D, D)
    x = [_dev(t, "bf16") for t in a]
    op.set_seq_lengths(first)
    op.forward(*x, train=False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, sT = op.forward(*x, train=False)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        _delay()
        graph.replay()
        kept = o.clone(), sT.clone()
        op.set_seq_lengths(second)
        graph.replay()
    torch.cuda.synchronize()
    for lens, (oo, ss) in zip((first, second), (kept, (o, sT))):
        wo, ws, _ = O.delta_forward(*a, None, lens)
        _close(_host(oo), wo, TOL["bf16"], f"o of lengths {lens}")
        _close(_host(ss), ws, STATE_TOL["bf16"], f"state of lengths {lens}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_later_call_on_another_stream_keeps_the_reserve(dtype):
    """A training forward queued on one stream does not overwrite what a backward still waiting on another reads."""
    import torch
    import bwd_persistent_cta_gb300 as R
    shape = (90, 2, 1, 2, 64, 64)
    one, two = _inputs(*shape, dtype, 404), _inputs(*shape, dtype, 405)
    op = R.DeltaRule(2, 90, 1, 2, 64, 64, dtype=dtype)
    x1, x2 = ([_dev(i[n], dtype) for n in NAMES] for i in (one, two))
    do = _dev(one["do"], dtype)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    op.forward(*x1)
    op.backward(do, *x1)
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        op.forward(*x1)
        _delay()
        grads = op.backward(do, *x1)
    with torch.cuda.stream(s2):
        op.forward(*x2)
    torch.cuda.synchronize()
    a = [one[n] for n in NAMES]
    o, sT, kept = O.delta_forward(*a)
    want = O.delta_backward(one["do"], *a, sT, kept)
    for name, g, w in zip(("dq", "dk", "dv", "dg", "dbeta"), grads, want):
        _close(_host(g), w, TOL[dtype], name)


def test_norm_gradients_on_two_streams_run_in_order():
    """Two backward calls of one handle share its scratch, so the second waits for the first."""
    import torch
    import bwd_persistent_cta_gb300 as R
    op = R.BlockNorm(64, 256)
    y, w = torch.randn(64, 256, device="cuda").bfloat16(), torch.ones(256, device="cuda").bfloat16()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    op.backward(y, None, y, w_in=w)
    torch.cuda.synchronize()
    first, second = torch.cuda.Event(), torch.cuda.Event()
    with torch.cuda.stream(s1):
        _delay()
        op.backward(y, None, y, w_in=w)
        first.record()
    with torch.cuda.stream(s2):
        op.backward(y, None, y, w_in=w)
        second.record()
    second.synchronize()
    assert first.query()


def _busy_block(like):
    """A block of the current stream's pool that the stream still reads although the host has dropped it, and where the
    reading ends up."""
    import torch
    x = torch.full_like(like, 3.0)
    torch.cuda.synchronize()
    _delay()
    return x.clone()


def test_outputs_on_a_stream_that_is_not_current():
    """With ``stream=``, outputs do not take memory that the current stream has yet to read."""
    import torch
    import bwd_persistent_cta_gb300 as R
    s = torch.cuda.Stream()
    T, B, H, D = 256, 8, 16, 128                 # 8 MB: blocks of their own
    op = R.DeltaRule(B, T, H, H, D, D)
    x = [_dev(t, "bf16") for t in (_inputs(T, B, H, H, D, D, "bf16", 406)[n] for n in NAMES)]
    norm = R.BlockNorm(B * T, H * D)
    one = R.DeltaRule(B, 1, H, H, D, D)
    st = torch.zeros(B, H, D, D, device="cuda")
    flat = x[2].view(B * T, H * D)
    calls = [
        (x[2], lambda: op.forward(*x, train=False, stream=s)),
        (flat, lambda: norm.forward(flat, stream=s)),
        (x[2], lambda: (op.forward(*x, stream=s), op.backward(x[2], *x, stream=s))),
        (flat, lambda: norm.backward(flat, None, flat, stream=s)),
        (x[2][:1].contiguous(), lambda: one.step(*(t[:1].contiguous() for t in x), st, stream=s)),
    ]
    for like, call in calls:
        call()
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        kept = _busy_block(like)
        out = call()
        torch.cuda.synchronize()
        assert torch.all(kept == 3.0)
        del out


def test_outputs_dropped_while_the_current_stream_reads_them():
    import torch
    import bwd_persistent_cta_gb300 as R
    s = torch.cuda.Stream()
    rows, cols = 2048, 2048
    op = R.BlockNorm(rows, cols)
    y = torch.randn(rows, cols, device="cuda").bfloat16()
    zero = torch.zeros_like(y)
    want, _ = op.forward(y)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    out, _ = op.forward(y, stream=s)
    torch.cuda.synchronize()
    _delay()
    kept = out.clone()
    del out
    again, _ = op.forward(zero, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(kept, want)


def test_inputs_dropped_while_another_stream_reads_them():
    import torch
    import bwd_persistent_cta_gb300 as R
    s = torch.cuda.Stream()
    rows, cols = 2048, 2048
    op = R.BlockNorm(rows, cols)
    y = torch.randn(rows, cols, device="cuda").bfloat16()
    want, _ = op.forward(y)
    op.forward(y, stream=s)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        _delay()
    out, _ = op.forward(y, stream=s)
    del y
    others = [torch.zeros(rows, cols, device="cuda", dtype=torch.bfloat16) for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(out, want) and not any(t.any() for t in others)


def test_a_stream_of_another_device_is_refused():
    import torch
    import bwd_persistent_cta_gb300 as R

    class Other:
        device, cuda_stream = torch.device("cuda", 7), 0

    op = R.BlockNorm(4, 64)
    y = torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="stream"):
        op.forward(y, stream=Other())
