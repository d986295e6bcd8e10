"""SelectiveScan, CausalConv and GradClip over more than 2^31 elements: what lies behind
them equals the same tokens, slots or elements by themselves."""
import pytest

pytestmark = pytest.mark.gpu

T, D = (1 << 19) + 77, 4104            # 2.15e9 elements of one sequence
LAST = 131


@pytest.fixture(autouse=True)
def _memory():
    import torch
    if torch.cuda.get_device_properties(0).total_memory < 120e9:
        pytest.skip("needs 100 GB")
    yield
    torch.cuda.empty_cache()


def _bf16(*shape, seed=1):
    """Values between -1 and 1, made where they are used."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
    return out.uniform_(-1, 1, generator=gen)


def test_convolution_of_a_long_sequence():
    import torch
    import bwd_persistent_cta_gb300 as R
    assert T * D > 1 << 31
    x, dy, w = _bf16(T, 1, D), _bf16(T, 1, D, seed=2), _bf16(D, 4, seed=3)
    op, end = R.CausalConv(1, T, D, 4), R.CausalConv(1, LAST, D, 4)
    y, sT = op.forward(x, w)
    d = op.backward(dy, x, w)
    s0 = x[T - LAST - 3:T - LAST].transpose(0, 1).contiguous()
    y2, s2 = end.forward(x[-LAST:], w, s0=s0)
    d2 = end.backward(dy[-LAST:], x[-LAST:], w, s0=s0)
    assert torch.equal(y[-LAST:], y2) and torch.equal(sT, s2) and torch.equal(d["dx"][-LAST:], d2["dx"])
    # the weights' gradients are the two parts'
    first = R.CausalConv(1, T - LAST, D, 4)
    d1 = first.backward(dy[:-LAST], x[:-LAST], w)
    assert ((d["dw"] - (d1["dw"] + d2["dw"])).norm() <= 2e-5 * d["dw"].norm()).item()


def test_scan_of_a_long_sequence():
    import torch
    import bwd_persistent_cta_gb300 as R
    N = 8
    x, dt, dy = _bf16(T, 1, D), _bf16(T, 1, D, seed=2), _bf16(T, 1, D, seed=3)
    B, C = _bf16(T, 1, 1, N, seed=4), _bf16(T, 1, 1, N, seed=5)
    A, bias = -torch.arange(1.0, N + 1, device="cuda").repeat(D, 1), torch.full((D,), -3.0, device="cuda")
    op, first, end = (R.SelectiveScan(1, n, D, N) for n in (T, T - LAST, LAST))
    y, hT = op.forward(x, dt, A, B, C, dt_bias=bias)
    d = op.backward(dy, x, dt, A, B, C, dt_bias=bias)
    cut = lambda a, b: [t if t is A else t[a:b] for t in (x, dt, A, B, C)]  # noqa: E731
    _, h0 = first.forward(*cut(0, T - LAST), dt_bias=bias, train=False)
    y2, h2 = end.forward(*cut(T - LAST, T), dt_bias=bias, h0=h0)
    d2 = end.backward(dy[-LAST:], *cut(T - LAST, T), dt_bias=bias)
    # the same sums in pieces of other lengths: fp32 states to 1e-5, bf16 results to a rounding
    pairs = [(hT, h2, 1e-5), (y[-LAST:], y2, 2.0 ** -8)]
    pairs += [(d[n][-LAST:], d2[n], 2.0 ** -8) for n in ("dx", "ddt", "dB", "dC")]
    for a, b, tol in pairs:
        assert ((a.float() - b.float()).norm() <= tol * b.float().norm()).item()
    assert all(torch.isfinite(d[n].sum()).item() for n in ("dA", "ddt_bias", "dh0"))


def test_steps_against_a_large_pool():
    import torch
    import bwd_persistent_cta_gb300 as R
    slots, D, N = 33000, 4096, 16
    assert slots * D * N > 1 << 31
    pool = torch.zeros(slots, D, N, device="cuda")
    pool[-1] = 1.0
    pool[3] = 2.0
    B, C = _bf16(1, 2, 1, N, seed=4), _bf16(1, 2, 1, N, seed=5)
    x, dt, A = _bf16(1, 2, D), _bf16(1, 2, D, seed=2), -torch.ones(D, N, device="cuda")
    small = torch.stack([pool[-1], pool[3]])
    op = R.SelectiveScan(2, 1, D, N)
    at = torch.tensor([slots - 1, 3], dtype=torch.int32, device="cuda")
    y, want = op.step(x, dt, A, B, C, pool, slots=at), op.step(x, dt, A, B, C, small)
    assert torch.equal(y, want) and torch.equal(pool[-1], small[0]) and torch.equal(pool[3], small[1])
    assert not pool[:3].any() and not pool[4:-1].any()
    slots, D = 180000, 4096
    assert slots * D * 3 > 1 << 31
    pool = torch.zeros(slots, 3, D, device="cuda", dtype=torch.bfloat16)
    pool[-1] = 1.0
    conv, w = R.CausalConv(2, 1, D, 4), _bf16(D, 4, seed=6)
    small = torch.stack([pool[-1], pool[3]])
    at = torch.tensor([slots - 1, 3], dtype=torch.int32, device="cuda")
    y, want = conv.step(x, w, pool, slots=at), conv.step(x, w, small)
    assert torch.equal(y, want) and torch.equal(pool[-1], small[0]) and torch.equal(pool[3], small[1])
    assert not pool[:3].any() and not pool[4:-1].any()


@pytest.mark.parametrize("inplace", [True, False])
def test_clipping_a_large_tensor(inplace):
    import torch
    import bwd_persistent_cta_gb300 as R
    n = (1 << 31) + 12345
    g, small = torch.full((n,), 0.5, device="cuda", dtype=torch.bfloat16), torch.full((77,), 3.0, device="cuda")
    g[-1] = 64.0
    out = None if inplace else [torch.zeros_like(g), torch.zeros_like(small)]
    norm = R.GradClip([n, 77], ["bf16", "f32"]).clip([g, small], 1.0, eps=0.0, out=out).item()
    want = (0.25 * (n - 1) + 64.0 ** 2 + 77 * 9.0) ** 0.5
    assert abs(norm - want) <= 2.0 ** -22 * want
    a, b = (g, small) if inplace else out
    half = torch.tensor(0.5 / want).bfloat16().item()
    assert abs(a[-1].item() - 64 / want) <= 2.0 ** -8 * 64 / want and abs(b[0].item() - 3 / want) <= 2.0 ** -21 * 3 / want
    # every other element is one and the same number
    assert a[:-1].min().item() == a[:-1].max().item() and abs(a[0].item() - half) <= 2.0 ** -8 * half
