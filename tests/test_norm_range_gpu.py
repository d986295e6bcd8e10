"""The block norm's gradients on rows far from unit size: the inverse root mean
enters them in the third power, which leaves the range of fp32 long before the
gradient itself does."""
import numpy as np
import pytest

from oracle import lm_oracle as O

from tests.test_norm_gpu import TOL, _close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e-16, 1e-13, 1e13, 1e16])
def test_gradients_of_small_and_large_rows(size, dtype):
    """Both norms, each row to the tolerance of whole tensors."""
    import torch
    import bwd_persistent_cta_gb300 as R
    rows, cols, eps = 4, 256, 1e-38
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator().manual_seed(601)
    rnd = lambda: torch.randn(rows, cols, generator=gen)  # noqa: E731
    y, x = (size * rnd()).to(td), (size * rnd()).to(td)
    d, dn = (rnd() / size).to(td), rnd().to(td)
    h = lambda t: t.double().numpy()  # noqa: E731

    op = R.BlockNorm(rows, cols, dtype=dtype, eps=eps)
    g = op.backward(dn.cuda(), None, y.cuda())
    _, _, saved = O.norm_forward(h(y), eps=eps)
    want = O.norm_backward(h(dn), None, h(y), saved)
    for r in range(rows):
        _close(h(g["dy"].cpu())[r], want["dy"][r], TOL[dtype], "dy")

    op = R.BlockNorm(rows, cols, dtype=dtype, norm_in=False, residual=True, norm_out=True, eps=eps)
    g = op.backward(d.cuda(), dn.cuda(), y.cuda(), x=x.cuda())
    _, _, saved = O.norm_forward(h(y), x=h(x), norm_in=False, norm_out=True, eps=eps)
    want = O.norm_backward(h(d), h(dn), h(y), saved, x=h(x), norm_in=False)
    for n in ("dy", "dx"):
        for r in range(rows):
            _close(h(g[n].cpu())[r], want[n][r], TOL[dtype], n)


def test_gradient_of_a_zero_row():
    """A row of zeros has the gradient of y / sqrt(eps), whatever eps."""
    import torch
    import bwd_persistent_cta_gb300 as R
    for eps in (1e-6, 1e-30):
        op = R.BlockNorm(1, 64, dtype="f32", eps=eps)
        d = torch.linspace(-1, 1, 64).view(1, 64)
        g = op.backward(d.cuda(), None, torch.zeros(1, 64, device="cuda"))["dy"].cpu().double().numpy()
        _close(g, d.double().numpy() / np.sqrt(eps), TOL["f32"], f"eps {eps}")
