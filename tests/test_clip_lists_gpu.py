"""Which lists of tensors clipping takes."""
import pytest

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
