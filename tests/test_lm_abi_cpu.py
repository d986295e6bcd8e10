"""The boundary of the gated delta rule and the block norm without a GPU:
descriptors refused before any device call, NULL and misaligned arguments,
structs equal to the header's, and the wrappers' tensor checks."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def R():
    from bwd_persistent_cta_gb300 import build
    build.build()
    import bwd_persistent_cta_gb300 as R
    R.lib()
    return R


def _fields(name):
    txt = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "rnn.h")).read(), flags=re.S)
    body = re.search(r"typedef struct\s*\{([^{}]*)\}\s*" + name + r"\s*;", txt).group(1)
    out = []
    for decl in filter(None, (d.strip() for d in body.split(";"))):
        kind, names = re.match(r"(const void\*|int64_t|int|float)\s+(.*)", decl, flags=re.S).groups()
        out += [(n.strip(), kind) for n in names.split(",")]
    return out


@pytest.mark.parametrize("name", ["rnn_delta_desc_t", "rnn_delta_in_t", "rnn_norm_desc_t", "rnn_norm_in_t"])
def test_structs_match_header(R, name):
    kinds = {"int": ctypes.c_int, "float": ctypes.c_float, "int64_t": ctypes.c_int64, "const void*": ctypes.c_void_p}
    assert [(n, kinds[k]) for n, k in _fields(name)] == list(getattr(R, name)._fields_)


def _delta(R, **kw):
    d = dict(batch=2, seq_len=5, heads_k=2, heads_v=4, dim_k=64, dim_v=64, dtype=R.RNN_BF16, batch_first=0, scale=0.0)
    d.update(kw)
    return R.rnn_delta_desc_t(**d)


def _norm(R, **kw):
    d = dict(rows=4, groups=2, cols=64, dtype=R.RNN_BF16, norm_in=1, gate=1, residual=1, norm_out=1, eps=1e-6)
    d.update(kw)
    return R.rnn_norm_desc_t(**d)


BAD_DELTA = [dict(batch=0), dict(seq_len=0), dict(heads_k=0), dict(heads_v=3), dict(heads_v=0), dict(dim_k=4),
             dict(dim_k=12), dict(dim_k=264), dict(dim_v=0), dict(dim_v=20), dict(dim_v=512), dict(dtype=2),
             dict(batch_first=2), dict(scale=float("nan")), dict(scale=float("inf")),
             dict(batch=1 << 15, seq_len=1 << 16), dict(batch=1 << 20, heads_k=1 << 10, heads_v=1 << 10)]
BAD_NORM = [dict(rows=0), dict(groups=0), dict(rows=1 << 20, groups=1 << 11), dict(cols=4), dict(cols=12),
            dict(cols=8200), dict(dtype=-1), dict(norm_in=2), dict(gate=3), dict(gate=-1), dict(residual=-1),
            dict(norm_out=5), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))]


@pytest.mark.parametrize("kw", BAD_DELTA, ids=str)
def test_bad_delta_descriptor(R, kw):
    h = ctypes.c_void_p(16)
    assert R.lib().rnn_delta_create(ctypes.byref(_delta(R, **kw)), ctypes.byref(h)) == R.RNN_BAD_PARAM
    assert not h.value


@pytest.mark.parametrize("kw", BAD_NORM, ids=str)
def test_bad_norm_descriptor(R, kw):
    h = ctypes.c_void_p(16)
    assert R.lib().rnn_norm_create(ctypes.byref(_norm(R, **kw)), ctypes.byref(h)) == R.RNN_BAD_PARAM
    assert not h.value


@pytest.mark.skipif(os.path.exists("/dev/nvidia0"), reason="checks the no-device path")
def test_create_without_device_fails_cleanly(R):
    h = ctypes.c_void_p(16)
    assert R.lib().rnn_delta_create(ctypes.byref(_delta(R)), ctypes.byref(h)) in (R.RNN_CUDA_ERROR, R.RNN_NOT_SUPPORTED)
    assert not h.value
    assert R.lib().rnn_norm_create(ctypes.byref(_norm(R)), ctypes.byref(h)) in (R.RNN_CUDA_ERROR, R.RNN_NOT_SUPPORTED)
    assert not h.value


def test_null_arguments(R):
    L, bad = R.lib(), R.RNN_BAD_PARAM
    h = ctypes.c_void_p()
    assert L.rnn_delta_create(None, ctypes.byref(h)) == bad and L.rnn_norm_create(None, ctypes.byref(h)) == bad
    assert L.rnn_delta_create(ctypes.byref(_delta(R)), None) == bad
    assert L.rnn_norm_create(ctypes.byref(_norm(R)), None) == bad
    assert L.rnn_delta_destroy(None) == R.RNN_OK and L.rnn_norm_destroy(None) == R.RNN_OK
    assert L.rnn_delta_get_sizes(None, None, None, None) == bad and L.rnn_norm_get_sizes(None, None) == bad
    assert L.rnn_delta_set_seq_lengths(None, None) == bad
    assert L.rnn_delta_forward(None, None, *([None] * 6)) == bad
    assert L.rnn_delta_backward(None, None, *([None] * 11)) == bad
    assert L.rnn_delta_step(None, None, None, 1, None, None, None) == bad
    assert L.rnn_norm_forward(None, None, *([None] * 3)) == bad
    assert L.rnn_norm_backward(None, None, *([None] * 10)) == bad
    assert L.rnn_delta_launch_count(None) == 0 and L.rnn_norm_launch_count(None) == 0


@pytest.mark.parametrize("kw", [dict(dtype="fp16"), dict(dtype="bfloat16")])
def test_wrappers_reject_bad_dtype(R, kw):
    with pytest.raises(ValueError):
        R.DeltaRule(1, 1, 1, 1, 64, 64, **kw)
    with pytest.raises(ValueError):
        R.BlockNorm(1, 64, **kw)


def test_norm_wrapper_rejects_unknown_gate(R):
    with pytest.raises(ValueError, match="gate"):
        R.BlockNorm(1, 64, gate="relu")


def _unbound(R, cls, desc):
    """A wrapper without a handle on the CPU device: its checks run before any library call."""
    import torch
    w = object.__new__(cls)
    w.torch, w.device, w.tdtype, w.desc, w.handle = torch, torch.device("cpu"), torch.bfloat16, desc, None
    w._shapes()
    return w


@pytest.mark.parametrize("bfirst", [0, 1])
def test_delta_wrapper_rows(R, bfirst):
    import torch
    op = _unbound(R, R.DeltaRule, _delta(R, batch_first=bfirst))
    lead = (2, 5) if bfirst else (5, 2)
    bf = torch.bfloat16
    packed = torch.zeros(*lead, 2 * 128 + 256, dtype=bf)
    q, k, v = packed.split([128, 128, 256], -1)
    q, k, v = q.unflatten(-1, (2, 64)), k.unflatten(-1, (2, 64)), v.unflatten(-1, (4, 64))
    gates = torch.zeros(*lead, 8, dtype=bf)
    g, beta = gates.split([4, 4], -1)
    x = op._inputs(q, k, v, g, beta)
    assert (x.q_row, x.k_row, x.v_row, x.g_row, x.beta_row) == (512, 512, 512, 8, 8)
    x = op._inputs(q.contiguous(), k.contiguous(), v.contiguous(), g.contiguous(), beta.contiguous())
    assert (x.q_row, x.k_row, x.v_row, x.g_row, x.beta_row) == (128, 128, 256, 4, 4)
    bad = [
        lambda: op._inputs(q[..., :1, :], k, v, g, beta),                               # heads
        lambda: op._inputs(q.transpose(0, 1), k, v, g, beta),                           # order of batch and time
        lambda: op._inputs(q.float(), k, v, g, beta),                                   # dtype
        lambda: op._inputs(q, k, v, g.float(), beta),
        lambda: op._inputs(q.contiguous().transpose(-1, -2).contiguous().transpose(-1, -2), k, v, g, beta),
        lambda: op._inputs(q, k, v[..., :32], g, beta),                                 # width
        lambda: op._inputs(torch.zeros(lead[0] + 1, lead[1] + 1, 2, 64, dtype=bf)[:-1, :-1], k, v, g, beta),  # two strides
        lambda: op._inputs(torch.zeros(1, 1, 2, 64, dtype=bf).expand(*lead, 2, 64), k, v, g, beta),           # overlap
        lambda: op._inputs(torch.zeros(*lead, 132, dtype=bf)[..., 4:].unflatten(-1, (2, 64)), k, v, g, beta),  # alignment
        lambda: op._inputs([0.0], k, v, g, beta),
    ]
    for f in bad:
        with pytest.raises((ValueError, TypeError)):
            f()


def test_delta_wrapper_checks_states(R):
    import torch
    op = _unbound(R, R.DeltaRule, _delta(R))
    bf = torch.bfloat16
    x = [torch.zeros(5, 2, 2, 64, dtype=bf)] * 2 + [torch.zeros(5, 2, 4, 64, dtype=bf)] + [torch.zeros(5, 2, 4, dtype=bf)] * 2
    with pytest.raises(ValueError, match="state"):
        op.step(*x, torch.zeros(4, 64, 64))
    with pytest.raises(ValueError, match="state"):
        op.step(*x, torch.zeros(3, 4, 64, 32))
    with pytest.raises(ValueError, match="state"):
        op.step(*x, torch.zeros(3, 4, 64, 64, dtype=bf))
    with pytest.raises(ValueError, match="slots"):
        op.step(*x, torch.zeros(1, 4, 64, 64))
    with pytest.raises(ValueError, match="slots"):
        op.step(*x, torch.zeros(3, 4, 64, 64), slots=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="s0"):
        op.forward(*x, s0=torch.zeros(2, 4, 64, 32))
    with pytest.raises(ValueError, match="training forward"):
        op.backward(x[2], *x)
    with pytest.raises(ValueError, match="one length"):
        op.set_seq_lengths([1])


def test_norm_wrapper_checks(R):
    import torch
    op = _unbound(R, R.BlockNorm, _norm(R))
    bf = torch.bfloat16
    y = torch.zeros(4, 128, dtype=bf)
    w = torch.ones(64, dtype=bf)
    wide = torch.zeros(4, 256, dtype=bf)[:, 128:]
    a = op._inputs(y, wide, y, w, None, w)
    assert (a.y_row, a.z_row, a.x_row) == (128, 256, 128) and a.scale is None
    for kw in (dict(z=None), dict(x=None), dict(w_in=torch.ones(128, dtype=bf)), dict(w_out=w.float()),
               dict(y=y[:, ::2]), dict(y=y[:2]), dict(z=torch.zeros(4, 257, dtype=bf)[:, 1:129])):
        with pytest.raises(ValueError):
            op._inputs(**{**dict(y=y, z=wide, x=y, w_in=w, scale=w, w_out=w), **kw})
    with pytest.raises(ValueError, match="required"):
        op.backward(None, None, y, wide, y)
    plain = _unbound(R, R.BlockNorm, _norm(R, gate=0, residual=0, norm_out=0))
    for kw in (dict(z=y), dict(x=y), dict(scale=w), dict(w_out=w)):
        with pytest.raises(ValueError, match="not used"):
            plain.forward(y, **kw)
    with pytest.raises(ValueError, match="not used"):
        plain.backward(y, y, y)
