"""Gradient clipping on the GPU against the fp64 reference: lists of any number of
tensors of any size and alignment, both types mixed, values over the whole range.

Tolerances, derived before the first run: the norm 2^-22 (sums of a few squares in
fp32, added in 64 bits, a root and a rounding: below 3 * 2^-24); scaled values 2^-22 in
fp32 (norm, sum with eps, quotient, product: four roundings) and 2^-8 each in bf16, half
a step (2^-9) and as much for the factor's own error beside a border."""
import numpy as np
import pytest

from oracle import ssm_oracle as O

pytestmark = pytest.mark.gpu


def _tensors(counts, dtypes, seed, scale=1.0, flat=False):
    import torch
    gen = torch.Generator().manual_seed(seed)
    td = {"f32": torch.float32, "bf16": torch.bfloat16}
    vals = [(scale * torch.randn(n, generator=gen)).to(td[d]) for n, d in zip(counts, dtypes)]
    if not flat:
        return [v.cuda() for v in vals]
    out = []                                       # slices of one buffer for each type, end to end
    for d in ("f32", "bf16"):
        buf = torch.cat([v for v, e in zip(vals, dtypes) if e == d] or [torch.empty(0, dtype=td[d])]).cuda()
        out.append(list(buf.split([v.numel() for v, e in zip(vals, dtypes) if e == d])))
    return [out[0 if d == "f32" else 1].pop(0) for d in dtypes]


def check(tensors, max_norm, eps=1e-6, inplace=True, dtypes=None):
    import torch
    import bwd_persistent_cta_gb300 as R
    host = [t.double().cpu().numpy() for t in tensors]
    norm, want = O.clip(host, max_norm, eps)
    op = R.GradClip([t.numel() for t in tensors], ["f32" if t.dtype == torch.float32 else "bf16" for t in tensors])
    alone = op.norm(tensors)
    out = None if inplace else [torch.full_like(t, float("nan")) for t in tensors]
    got = op.clip(tensors, max_norm, eps=eps, out=out)
    torch.cuda.synchronize()
    assert torch.equal(alone, got)
    # a subnormal norm is a multiple of 2^-149: its rounding alone is half of that
    assert abs(got.item() - norm) <= 2.0 ** -22 * norm + 2.0 ** -150
    for t, w, h in zip(tensors if inplace else out, want, host):
        g = t.double().cpu().numpy()
        tol = 2.0 ** -22 if t.dtype == torch.float32 else 2.0 ** -8
        assert np.all(np.abs(g - w) <= tol * np.abs(w) + (2.0 ** -149 if t.dtype == torch.float32 else 2.0 ** -133))
        if np.array_equal(w, h):
            assert np.array_equal(g, h)
    if not inplace:
        for t, h in zip(tensors, host):
            assert np.array_equal(t.double().cpu().numpy(), h)
    return op


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 255, 2047, 2048, 2049, 100003])
@pytest.mark.parametrize("inplace", [True, False])
def test_one_tensor(n, dtype, inplace):
    check(_tensors([n], [dtype], n), 0.5, inplace=inplace)
    check(_tensors([n], [dtype], n), 1e9, inplace=inplace)


@pytest.mark.parametrize("flat", [False, True])
@pytest.mark.parametrize("inplace", [True, False])
def test_many_tensors_of_both_types(flat, inplace):
    counts = [0, 1, 5000, 3, 64, 0, 70001, 7, 129, 40000, 1, 0]
    dtypes = ["f32", "bf16", "bf16", "f32", "f32", "bf16", "f32", "bf16", "bf16", "f32", "f32", "f32"]
    check(_tensors(counts, dtypes, 1, flat=flat), 1.0, inplace=inplace)


@pytest.mark.parametrize("num", [100, 101, 999, 1000, 1001, 2500])
def test_long_lists(num):
    counts = [(i * 37) % 90 for i in range(num)]
    check(_tensors(counts, ["bf16" if i % 3 else "f32" for i in range(num)], 2, flat=True), 1.0)


def test_shapes_and_large():
    import torch
    t = [torch.randn(300, 7, 11, device="cuda"), torch.randn(4096, 4099, device="cuda"),
         torch.randn(5, 5, device="cuda").bfloat16()]
    check([x.view(-1) for x in t], 2.0)
    import bwd_persistent_cta_gb300 as R
    op = R.GradClip([x.numel() for x in t], ["f32", "f32", "bf16"])
    assert abs(op.clip(t, 1.0).item() - 2.0) < 1e-4 and abs(op.norm(t).item() - 1.0) < 1e-4


@pytest.mark.parametrize("inplace", [True, False])
def test_offsets_differ_between_input_and_output(inplace):
    import torch
    import bwd_persistent_cta_gb300 as R
    for dtype, name in ((torch.float32, "f32"), (torch.bfloat16, "bf16")):
        for a, b in ((0, 1), (1, 0), (3, 3), (5, 2)):
            src, dst = torch.randn(3000, device="cuda").to(dtype), torch.zeros(3000, device="cuda", dtype=dtype)
            g, o = src[a:a + 2500], dst[b:b + 2500]
            op = R.GradClip([2500], name)
            norm = op.clip([g], 1.0, out=[o])
            want = (g.double() / (norm.double() + 1e-6)).cpu()
            tol = 2.0 ** -21 if dtype == torch.float32 else 2.0 ** -8
            assert ((o.double().cpu() - want).abs() <= tol * want.abs()).all()
            assert not dst[:b].any() and not dst[b + 2500:].any()


@pytest.mark.parametrize("scale", [1e-42, 1e-30, 1e-20, 1e18, 1e25, 1e36])
def test_values_over_the_whole_range(scale):
    """Squares leave fp32 long before the norm does."""
    for counts in ([17], [5000, 3, 20000]):
        check(_tensors(counts, ["f32"] * len(counts), 3, scale), scale, eps=0.0)


def test_large_beside_small():
    import torch
    t = [torch.cat([torch.full((1,), 1e30), torch.full((999,), 1e-30)]).cuda(), torch.full((5000,), 1e-25).cuda()]
    check(t, 1.0)
    check([torch.zeros(100).cuda(), torch.full((1,), 3e-40).cuda()], 1.0, eps=0.0)


def test_zeros():
    import torch
    import bwd_persistent_cta_gb300 as R
    t = [torch.zeros(1000, device="cuda"), torch.zeros(3, device="cuda").bfloat16()]
    op = R.GradClip([1000, 3], ["f32", "bf16"])
    for limit, eps in ((1.0, 1e-6), (0.0, 0.0), (0.0, 1e-6)):
        assert op.clip(t, limit, eps=eps).item() == 0 and not t[0].any() and not t[1].any()
    t[0][5] = 2.0
    assert op.clip(t, 0.0).item() == 2.0 and not t[0].any()
    empty = R.GradClip([0, 0])
    assert empty.clip([t[0][:0], t[0][:0]], 1.0).item() == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_norm_that_is_not_finite_changes_nothing(bad):
    import torch
    import bwd_persistent_cta_gb300 as R
    t = [torch.randn(5000, device="cuda"), torch.randn(777, device="cuda").bfloat16()]
    t[1][700] = bad
    keep = [x.clone() for x in t]
    op = R.GradClip([5000, 777], ["f32", "bf16"])
    out = [torch.zeros_like(x) for x in t]
    for o in (None, out):
        norm = op.clip(t, 1.0, out=o)
        assert torch.isnan(norm).item() if bad != bad else norm.item() == float("inf")
        for x, k in zip(t if o is None else o, keep):
            assert torch.equal(x.nan_to_num(7.0), k.nan_to_num(7.0))


def test_same_inputs_same_bits():
    import torch
    import bwd_persistent_cta_gb300 as R
    t = _tensors([300000, 17, 5000], ["bf16", "f32", "f32"], 4)
    op = R.GradClip([300000, 17, 5000], ["bf16", "f32", "f32"])
    a, b = op.norm(t), op.norm(t)
    assert torch.equal(a, b)


def test_refusals():
    import torch
    import bwd_persistent_cta_gb300 as R
    op = R.GradClip([100, 0, 50], ["f32", "f32", "bf16"])
    bad = R.RNN_BAD_PARAM
    m = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    p, ws = m.data_ptr(), torch.empty(op.workspace_bytes, dtype=torch.uint8, device="cuda")

    def call(grads=(p, None, p + 1024), out=None, limit=1.0, eps=1e-6, norm=p + 2048, work=ws.data_ptr()):
        return R.rnn_clip_scale(op.handle, grads, out, limit, eps, norm, work)

    assert call() == R.RNN_OK
    for kw in (dict(grads=(p, None, None)), dict(grads=(p + 2, None, p + 1024)), dict(grads=(p, None, p + 1025)),
               dict(out=(None, None, p)), dict(out=(p + 1, None, p + 1024)), dict(limit=-1.0), dict(limit=float("nan")),
               dict(limit=float("inf")), dict(eps=-1.0), dict(eps=float("nan")), dict(norm=None), dict(norm=p + 2)):
        assert call(**kw) == bad, kw
    for kw in (dict(work=None), dict(work=ws.data_ptr() + 8)):
        assert call(**kw) == R.RNN_BAD_WORKSPACE, kw
    # memory that two tensors share is not written; the norm of such a list is still one
    for kw in (dict(grads=(p, None, p + 398)), dict(grads=(p, None, p)), dict(out=(p + 1024, None, p + 1022)),
               dict(out=(p + 1024, None, p + 1422))):
        assert call(**kw) == bad, kw
    assert call(grads=(p, None, p + 400)) == R.RNN_OK and call(grads=(p, None, p), out=(p, None, p + 1024)) == R.RNN_OK
    assert R.rnn_clip_norm(op.handle, (p, None, p), p + 2048, ws.data_ptr()) == R.RNN_OK
    assert R.rnn_clip_norm(op.handle, (p, None, None), p + 2048, ws.data_ptr()) == bad
    t = [torch.zeros(100, device="cuda"), torch.zeros(0, device="cuda"), torch.zeros(50, device="cuda").bfloat16()]
    for wrong in (t[:2], [t[0], t[1], t[2].float()], [t[0][:50], t[1], t[2]], [t[0], t[1], torch.zeros(50).bfloat16()],
                  [torch.zeros(200, device="cuda")[::2], t[1], t[2]], [1.0, t[1], t[2]]):
        with pytest.raises((ValueError, TypeError)):
            op.clip(wrong, 1.0)
        with pytest.raises((ValueError, TypeError)):
            op.clip(t, 1.0, out=wrong)
    torch.cuda.synchronize()
