"""The operators together, as examples/gated_delta_block.py composes them: prefill plus decoding equals the whole
sequence, the block's gradients are the derivatives of its forward, and training it lowers the loss."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("gated_delta_block", os.path.join(ROOT, "examples", "gated_delta_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _inputs(B, T, width, dtype):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(B, T, width, device="cuda", generator=gen).to(dtype)
    n = (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(dtype)
    return x, n


def test_prefill_then_decode_is_the_whole_sequence(ex):
    import torch
    B, T, cut, width = 2, 75, 70, 256
    x, n = _inputs(B, T, width, torch.bfloat16)
    whole = ex.GatedDeltaBlock(B, T, width, 2, 4, 64)
    pre = ex.GatedDeltaBlock(B, cut, width, 2, 4, 64, weights=whole.w)
    one = ex.GatedDeltaBlock(B, 1, width, 2, 4, 64, weights=whole.w)
    x1, n1, _ = whole.forward(x, n)
    _, _, state = pre.forward(x[:, :cut].contiguous(), n[:, :cut].contiguous())
    pool = torch.zeros(5, 4, 64, 64, device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    pool[slots.long()] = state
    for t in range(cut, T):
        y, m = one.decode(x[:, t:t + 1].contiguous(), n[:, t:t + 1].contiguous(), pool, slots)
        # bf16 roundings of two different orders of the same sums, a handful on the way: 8 * 2^-9
        for got, want in ((y, x1[:, t:t + 1]), (m, n1[:, t:t + 1])):
            d = (got.float() - want.float()).norm() / want.float().norm()
            assert d <= 8 * 2.0 ** -9, (t, d)


def test_block_gradients_are_derivatives(ex):
    """fp32 storage; central differences with h = 1e-2 along unit-RMS directions.  Truncation and the fp32 forward's
    rounding (2^-24 sqrt(sum of squares) / h) both stay below 1e-3 of the gradient's norm times the direction's."""
    import torch
    B, T, width = 2, 70, 64
    x, n = _inputs(B, T, width, torch.float32)
    blk = ex.GatedDeltaBlock(B, T, width, 1, 2, 64, dtype="f32")
    gen = torch.Generator(device="cuda").manual_seed(5)
    dx1, dn1 = (torch.randn(x.shape, device="cuda", generator=gen) for _ in range(2))
    blk.forward(x, n, train=True)
    dx, dn, dw = blk.backward(dx1, dn1)

    def loss(xi, ni):
        x1, n1, _ = blk.forward(xi, ni)
        return ((x1.double() * dx1.double()).sum() + (n1.double() * dn1.double()).sum()).item()

    h = 1e-2
    for name, grad in (("x", dx), ("n", dn)):
        d = torch.randn(x.shape, device="cuda", generator=gen)
        d /= d.norm()
        up = loss(x + h * d, n) if name == "x" else loss(x, n + h * d)
        dn_ = loss(x - h * d, n) if name == "x" else loss(x, n - h * d)
        want, got = (up - dn_) / (2 * h), (grad.double() * d.double()).sum().item()
        assert abs(got - want) <= 1e-3 * grad.double().norm().item(), name
    for name, w in blk.w.items():
        d = torch.randn(w.shape, device="cuda", generator=gen)
        d /= d.norm()
        keep = w.clone()
        w.copy_(keep + h * d)
        up = loss(x, n)
        w.copy_(keep - h * d)
        down = loss(x, n)
        w.copy_(keep)
        want, got = (up - down) / (2 * h), (dw[name].double() * d.double()).sum().item()
        assert abs(got - want) <= 2e-3 * dw[name].double().norm().item(), name


def test_example_runs(ex, capsys):
    ex.main()
    out = capsys.readouterr().out
    err = [float(line.rsplit(" ", 1)[1]) for line in out.splitlines() if "mean squared error" in line]
    assert len(err) >= 2 and err[-1] < err[0] and "decoded 8 tokens" in out
