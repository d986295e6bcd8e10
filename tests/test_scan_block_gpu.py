"""The operators together, as examples/selective_scan_block.py composes them: prefill plus decoding equals the whole
sequence, the block's gradients are the derivatives of its forward, and the example runs."""
import importlib.util
import os

import pytest

from tests.test_delta_block_gpu import _inputs

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("selective_scan_block", os.path.join(ROOT, "examples", "selective_scan_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_prefill_then_decode_is_the_whole_sequence(ex):
    import torch
    B, T, cut, width, D, N = 2, 75, 70, 256, 264, 16
    x, n = _inputs(B, T, width, torch.bfloat16)
    whole = ex.SelectiveScanBlock(B, T, width, D, N, 16)
    pre = ex.SelectiveScanBlock(B, cut, width, D, N, 16, weights=whole.w)
    one = ex.SelectiveScanBlock(B, 1, width, D, N, 16, weights=whole.w)
    x1, n1, _, _ = whole.forward(x, n)
    _, _, sT, hT = pre.forward(x[:, :cut].contiguous(), n[:, :cut].contiguous())
    conv_pool, pool = torch.zeros(5, 3, D, device="cuda", dtype=torch.bfloat16), torch.zeros(5, D, N, device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    conv_pool[slots.long()], pool[slots.long()] = sT, hT
    for t in range(cut, T):
        y, m = one.decode(x[:, t:t + 1].contiguous(), n[:, t:t + 1].contiguous(), conv_pool, pool, slots)
        # bf16 roundings of two different orders of the same sums, a handful on the way: 8 * 2^-9
        for got, want in ((y, x1[:, t:t + 1]), (m, n1[:, t:t + 1])):
            d = (got.float() - want.float()).norm() / want.float().norm()
            assert d <= 8 * 2.0 ** -9, (t, d)


@pytest.mark.parametrize("T", [70, 200])
def test_block_gradients_are_derivatives(ex, T):
    """fp32 storage; central differences with h = 1e-2 along unit directions.  Truncation (h^2 of a smooth function of
    unit-sized values) and the fp32 forward's rounding (2^-24 sqrt(sum of squares) / h) both stay below 1e-3 of the
    gradient's norm times the direction's; the weights' larger gradients get twice that."""
    import torch
    B, width, D, N = 2, 64, 72, 16
    x, n = _inputs(B, T, width, torch.float32)
    blk = ex.SelectiveScanBlock(B, T, width, D, N, 8, dtype="f32")
    gen = torch.Generator(device="cuda").manual_seed(5)
    dx1, dn1 = (torch.randn(x.shape, device="cuda", generator=gen) for _ in range(2))
    blk.forward(x, n, train=True)
    dx, dn, dw = blk.backward(dx1, dn1)

    def loss(xi, ni):
        x1, n1, _, _ = blk.forward(xi, ni)
        return ((x1.double() * dx1.double()).sum() + (n1.double() * dn1.double()).sum()).item()

    h = 1e-2
    for name, grad in (("x", dx), ("n", dn)):
        d = torch.randn(x.shape, device="cuda", generator=gen)
        d /= d.norm()
        up = loss(x + h * d, n) if name == "x" else loss(x, n + h * d)
        down = loss(x - h * d, n) if name == "x" else loss(x, n - h * d)
        want, got = (up - down) / (2 * h), (grad.double() * d.double()).sum().item()
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
    assert out.count("mean squared error") == 5 and "nan" not in out and "decoded 8 tokens" in out
