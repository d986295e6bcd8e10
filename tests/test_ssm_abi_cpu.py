"""The boundary of the selective scan, the causal convolution and gradient clipping
without a GPU: descriptors refused before any device call, NULL arguments, structs
equal to the header's, and the wrappers' tensor checks."""
import ctypes
import os
import re

import pytest

from tests.test_lm_abi_cpu import R, ROOT, _unbound  # noqa: F401  (R is a fixture)


@pytest.mark.parametrize("name", ["rnn_scan_desc_t", "rnn_scan_in_t", "rnn_scan_grad_t", "rnn_conv_desc_t", "rnn_conv_in_t"])
def test_structs_match_header(R, name):  # noqa: F811
    txt = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "rnn.h")).read(), flags=re.S)
    body = re.search(r"typedef struct\s*\{([^{}]*)\}\s*" + name + r"\s*;", txt).group(1)
    kinds = {"int": ctypes.c_int, "int64_t": ctypes.c_int64, "const void*": ctypes.c_void_p, "void*": ctypes.c_void_p}
    want = []
    for decl in filter(None, (d.strip() for d in body.split(";"))):
        kind, names = re.match(r"(const void\*|void\*|int64_t|int)\s+(.*)", decl, flags=re.S).groups()
        want += [(n.strip(), kinds[kind]) for n in names.split(",")]
    assert want == list(getattr(R, name)._fields_)


def _scan(R, **kw):  # noqa: F811
    d = dict(batch=2, seq_len=5, channels=32, states=16, groups=2, dtype=R.RNN_BF16, batch_first=0, softplus=1)
    return R.rnn_scan_desc_t(**{**d, **kw})


def _conv(R, **kw):  # noqa: F811
    d = dict(batch=2, seq_len=5, channels=32, width=4, dtype=R.RNN_BF16, batch_first=0, act=R.RNN_GATE_SILU)
    return R.rnn_conv_desc_t(**{**d, **kw})


SEQS = [dict(batch=0), dict(seq_len=0), dict(channels=0), dict(channels=4), dict(channels=12), dict(channels=65544),
        dict(batch=1 << 16, seq_len=1 << 15), dict(batch=1 << 20, channels=1 << 16), dict(dtype=2), dict(dtype=-1),
        dict(batch_first=2)]


@pytest.mark.parametrize("kw", SEQS + [dict(states=0), dict(states=4), dict(states=20), dict(states=72), dict(groups=0),
                                       dict(groups=3), dict(groups=8), dict(groups=-1), dict(softplus=2)], ids=str)
def test_bad_scan_descriptor(R, kw):  # noqa: F811
    h = ctypes.c_void_p(16)
    assert R.lib().rnn_scan_create(ctypes.byref(_scan(R, **kw)), ctypes.byref(h)) == R.RNN_BAD_PARAM
    assert not h.value


@pytest.mark.parametrize("kw", SEQS + [dict(width=1), dict(width=5), dict(act=2), dict(act=-1)], ids=str)
def test_bad_conv_descriptor(R, kw):  # noqa: F811
    h = ctypes.c_void_p(16)
    assert R.lib().rnn_conv_create(ctypes.byref(_conv(R, **kw)), ctypes.byref(h)) == R.RNN_BAD_PARAM
    assert not h.value


@pytest.mark.parametrize("counts,dtypes", [([], []), ([-1], [0]), ([(1 << 40) + 1], [0]), ([1 << 40] * 5, [1] * 5), ([1], [2]),
                                           ([1, 1], [0, -1]), ([0] * 65537, [0] * 65537)], ids=lambda v: str(v)[:20])
def test_bad_clip_list(R, counts, dtypes):  # noqa: F811
    h = ctypes.c_void_p(16)
    n = len(counts)
    rc = R.lib().rnn_clip_create(n, (ctypes.c_int64 * n)(*counts), (ctypes.c_int * n)(*dtypes), ctypes.byref(h))
    assert rc == R.RNN_BAD_PARAM and not h.value


@pytest.mark.skipif(os.path.exists("/dev/nvidia0"), reason="checks the no-device path")
def test_create_without_device_fails_cleanly(R):  # noqa: F811
    none = (R.RNN_CUDA_ERROR, R.RNN_NOT_SUPPORTED)
    h = ctypes.c_void_p(16)
    assert R.lib().rnn_scan_create(ctypes.byref(_scan(R)), ctypes.byref(h)) in none and not h.value
    assert R.lib().rnn_conv_create(ctypes.byref(_conv(R)), ctypes.byref(h)) in none and not h.value
    one = (ctypes.c_int64 * 1)(5), (ctypes.c_int * 1)(0)
    assert R.lib().rnn_clip_create(1, *one, ctypes.byref(h)) in none and not h.value


def test_null_arguments(R):  # noqa: F811
    L, bad = R.lib(), R.RNN_BAD_PARAM
    h = ctypes.c_void_p()
    assert L.rnn_scan_create(None, ctypes.byref(h)) == bad and L.rnn_conv_create(None, ctypes.byref(h)) == bad
    assert L.rnn_scan_create(ctypes.byref(_scan(R)), None) == bad and L.rnn_conv_create(ctypes.byref(_conv(R)), None) == bad
    one = (ctypes.c_int64 * 1)(5), (ctypes.c_int * 1)(0)
    assert L.rnn_clip_create(1, None, one[1], ctypes.byref(h)) == bad and L.rnn_clip_create(1, one[0], None, ctypes.byref(h)) == bad
    assert L.rnn_clip_create(1, *one, None) == bad
    for name in ("scan", "conv", "clip"):
        assert getattr(L, f"rnn_{name}_destroy")(None) == R.RNN_OK
        assert getattr(L, f"rnn_{name}_launch_count")(None) == 0
    assert L.rnn_scan_get_sizes(None, None, None, None) == bad and L.rnn_conv_get_sizes(None, None) == bad
    assert L.rnn_clip_get_sizes(None, None) == bad
    assert L.rnn_scan_set_seq_lengths(None, None) == bad and L.rnn_conv_set_seq_lengths(None, None) == bad
    assert L.rnn_scan_forward(None, None, *([None] * 6)) == bad
    assert L.rnn_scan_backward(None, None, None, None, None, *([None] * 3)) == bad
    assert L.rnn_scan_step(None, None, None, 1, None, None, None) == bad
    assert L.rnn_conv_forward(None, None, *([None] * 4)) == bad
    assert L.rnn_conv_backward(None, None, *([None] * 9)) == bad
    assert L.rnn_conv_step(None, None, None, 1, None, None, None) == bad
    assert L.rnn_clip_scale(None, None, None, 1.0, 0.0, None, None, None) == bad
    assert L.rnn_clip_norm(None, None, None, None, None) == bad


def test_wrappers_reject_bad_names(R):  # noqa: F811
    with pytest.raises(ValueError, match="dtype"):
        R.SelectiveScan(1, 1, 8, 16, dtype="fp16")
    with pytest.raises(ValueError, match="dtype"):
        R.CausalConv(1, 1, 8, dtype="half")
    with pytest.raises(ValueError, match="act"):
        R.CausalConv(1, 1, 8, act="relu")
    with pytest.raises(ValueError, match="dtypes"):
        R.GradClip([1], ["fp16"])
    with pytest.raises(ValueError, match="one dtype"):
        R.GradClip([1, 2], ["f32"])


@pytest.mark.parametrize("bfirst", [0, 1])
def test_scan_wrapper_checks(R, bfirst):  # noqa: F811
    import torch
    op = _unbound(R, R.SelectiveScan, _scan(R, batch_first=bfirst))
    bf, f32 = torch.bfloat16, torch.float32
    lead = (2, 5) if bfirst else (5, 2)
    xz = torch.zeros(*lead, 64, dtype=bf)
    x, z = xz.split(32, -1)
    dbc = torch.zeros(*lead, 3 + 64, dtype=bf)
    _, B, C = dbc.split([3, 32, 32], -1)
    B, C = B.unflatten(-1, (2, 16)), C.unflatten(-1, (2, 16))
    dt, A, D = torch.zeros(*lead, 32, dtype=bf), torch.zeros(32, 16), torch.zeros(32)
    good = dict(x=x, dt=dt, A=A, B=B, C=C, z=z, D=D, dt_bias=D)
    a = op._inputs(**good)
    assert (a.x_row, a.dt_row, a.z_row, a.B_row, a.C_row) == (64, 32, 64, 67, 67)
    a = op._inputs(**{**good, "z": None, "D": None, "dt_bias": None})
    assert a.z is None and a.D is None and a.dt_bias is None
    for kw in (dict(x=None), dict(dt=None), dict(A=None), dict(B=None), dict(C=None), dict(x=x.float()), dict(x=x[..., :16]),
               dict(dt=torch.zeros(*lead, 33, dtype=bf)[..., 1:]), dict(A=A.to(bf)), dict(A=A.T.contiguous().T),
               dict(A=A[:, :8]), dict(D=D.to(bf)), dict(dt_bias=D[:8]), dict(B=B[..., :8]), dict(B=B.transpose(-1, -2)),
               dict(C=C[..., :1, :]), dict(z=z.transpose(0, 1)), dict(A=[0.0])):
        with pytest.raises((ValueError, TypeError)):
            op._inputs(**{**good, **kw})
    args = (x, dt, A, B, C)
    with pytest.raises(ValueError, match="training forward"):
        op.backward(x, *args)
    for st in (torch.zeros(4, 32), torch.zeros(3, 32, 8), torch.zeros(3, 32, 16, dtype=bf), torch.zeros(1, 32, 16)):
        with pytest.raises(ValueError, match="state"):
            op.step(*args, st)
    with pytest.raises(ValueError, match="slots"):
        op.step(*args, torch.zeros(3, 32, 16), slots=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="h0"):
        op.forward(*args, h0=torch.zeros(2, 32, 8))
    with pytest.raises(ValueError, match="y has"):
        op.forward(*args, y=torch.zeros(*lead, 32, dtype=f32))
    with pytest.raises(ValueError, match="one length"):
        op.set_seq_lengths([1])


def test_conv_wrapper_checks(R):  # noqa: F811
    import torch
    op = _unbound(R, R.CausalConv, _conv(R))
    bf = torch.bfloat16
    x = torch.zeros(5, 2, 64, dtype=bf)[..., :32]
    w, b = torch.zeros(32, 4, dtype=bf), torch.zeros(32, dtype=bf)
    assert op._inputs(x, w, b).x_row == 64 and op._inputs(x, w, None).bias is None
    for kw in (dict(x=None), dict(w=None), dict(x=x.float()), dict(w=w.float()), dict(w=w.T), dict(bias=b[:16]),
               dict(x=x[..., :16]), dict(bias=b.float())):
        with pytest.raises((ValueError, TypeError)):
            op._inputs(**{**dict(x=x, w=w, bias=b), **kw})
    with pytest.raises(ValueError, match="state"):
        op.step(x, w, torch.zeros(3, 4, 32, dtype=bf))
    with pytest.raises(ValueError, match="state"):
        op.step(x, w, torch.zeros(3, 3, 32))
    with pytest.raises(ValueError, match="s0"):
        op.forward(x, w, s0=torch.zeros(2, 3, 32))
    with pytest.raises(ValueError, match="dy"):
        op.backward(None, x, w)
    with pytest.raises(ValueError, match="one length"):
        op.set_seq_lengths([1, 2, 3])
