"""Which lists of tensors clipping takes, the flat weight gradient of recurrent layers among them."""
import numpy as np
import pytest

from oracle import ssm_oracle as O
from tests.test_lm_streams_gpu import _delay

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["values", "generator"])
def test_sequences_other_than_lists_on_another_stream(kind):
    """Gradients dropped while another stream has yet to read them are not reused, whatever held them."""
    import torch
    import bwd_persistent_cta_gb300 as R
    n = 1 << 22
    op = R.GradClip([n, n])
    g = {i: torch.full((n,), 2.0, device="cuda") for i in range(2)}
    out = {i: torch.zeros(n, device="cuda") for i in range(2)}
    op.clip(list(g.values()), 1.0, out=list(out.values()))
    want = [o.clone() for o in out.values()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        _delay()
    if kind == "values":
        op.clip(g.values(), 1.0, out=out.values(), stream=s)
    else:
        op.clip((v for v in g.values()), 1.0, out=(v for v in out.values()), stream=s)
    g.clear()
    others = [torch.zeros(n, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out.values(), want)) and not any(o.any() for o in others)
    g = {i: torch.full((n,), 2.0, device="cuda") for i in range(2)}
    with torch.cuda.stream(s):
        _delay()
    norm = op.norm(g.values() if kind == "values" else (v for v in g.values()), stream=s)
    g.clear()
    others = [torch.zeros(n, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert abs(norm.item() - 2.0 * (2 * n) ** 0.5) < 1e-2 and not any(o.any() for o in others)


def test_outputs_over_other_tensors_are_refused():
    """Each output is its own gradient or memory of its own, the norm too."""
    import torch
    import bwd_persistent_cta_gb300 as R
    op = R.GradClip([100, 0, 50], ["f32", "f32", "bf16"])
    m = torch.ones(8192, dtype=torch.uint8, device="cuda")
    p, ws = m.data_ptr(), torch.empty(op.workspace_bytes, dtype=torch.uint8, device="cuda")
    g = (p, None, p + 1024)

    def call(out, norm=p + 4096, grads=g):
        return R.rnn_clip_scale(op.handle, grads, out, 1.0, 1e-6, norm, ws.data_ptr())

    for out in (g, (p + 2048, None, p + 3584), (p, None, p + 2048), (p + 2048, p, p + 1024), (p + 400, None, p + 1124),
                (p + 2048, None, p + 924)):
        assert call(out) == R.RNN_OK, out
    # over the other gradient, over a shifted part of its own, and over both
    for out in ((p + 1024, None, p + 2048), (p + 2048, None, p), (p + 2048, None, p + 398), (p + 4, None, p + 1024),
                (p, None, p + 1026), (p + 1024, None, p), (p + 628, None, p + 2048), (p + 1120, None, p + 2048)):
        assert call(out) == R.RNN_BAD_PARAM, out
    for norm in (p, p + 396, p + 1024, p + 1120):
        assert call(None, norm) == R.RNN_BAD_PARAM and call((p + 2048, None, p + 3584), norm) == R.RNN_BAD_PARAM, norm
    for norm in (p + 2048, p + 3680):
        assert call((p + 2048, None, p + 3584), norm) == R.RNN_BAD_PARAM, norm
    assert call(None, p + 400) == R.RNN_OK and call(None, p + 1124) == R.RNN_OK
    # two gradients may share memory that is only read
    assert call((p + 2048, None, p + 3584), grads=(p, None, p + 200)) == R.RNN_OK
    torch.cuda.synchronize()


@pytest.mark.parametrize("num", [3, 1500])
def test_a_view_of_a_tensor_that_is_scaled_in_place(num):
    """Outputs elsewhere get the values from before, whichever CTA comes first."""
    import torch
    import bwd_persistent_cta_gb300 as R
    whole = torch.randn(3_000_000, device="cuda")
    rest = [torch.randn(5, device="cuda") for _ in range(num - 3)]
    keep = whole.clone()
    a, b = whole[7:1_500_007], whole[1_400_001:2_900_001]
    out = [whole, torch.empty_like(a), torch.empty_like(b)] + rest
    norm = R.GradClip([t.numel() for t in out]).clip([whole, a, b] + rest, 1.0, out=out)
    f = 1.0 / (norm.double().item() + 1e-6)
    for got, want in ((whole, keep), (out[1], keep[7:1_500_007]), (out[2], keep[1_400_001:2_900_001])):
        # the norm given back, its sum with eps, the factor and the product: four roundings
        assert ((got.double() - want.double() * f).abs() <= 2.0 ** -22 * f * want.double().abs()).all()


@pytest.mark.parametrize("mode,dtype", [("lstm", "bf16"), ("gru", "f32")])
def test_weight_gradients_of_recurrent_layers(mode, dtype):
    """The flat fp32 dw of a stack beside another operator's gradients, clipped in place."""
    import torch
    import bwd_persistent_cta_gb300 as R
    T, B, I, H = 12, 8, 40, 64
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    net = R.RNN(mode, I, H, T, B, num_layers=2, bidirectional=True, dtype=dtype)
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    w = (0.1 * rnd(net.weight_count)).to(td)
    x, dy = rnd(T, B, I).to(td), rnd(T, B, 2 * H).to(td)
    net.forward(x, w)
    net.backward_data(dy, w)
    dw = net.backward_weights(x)
    net.sync()
    other = rnd(333).bfloat16()
    host = [t.double().cpu().numpy() for t in (dw, other)]
    assert dw.dtype == torch.float32 and np.abs(host[0]).max() > 0
    limit = 0.25 * float(np.sqrt(sum((h ** 2).sum() for h in host)))
    norm, want = O.clip(host, float(np.float32(limit)))
    got = R.GradClip([dw.numel(), 333], ["f32", "bf16"]).clip([dw, other], limit)
    assert abs(got.item() - norm) <= 2.0 ** -22 * norm
    for t, v, tol in ((dw, want[0], 2.0 ** -22), (other, want[1], 2.0 ** -8)):
        assert np.all(np.abs(t.double().cpu().numpy() - v) <= tol * np.abs(v) + 2.0 ** -133)
