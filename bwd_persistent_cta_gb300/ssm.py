"""The selective scan, the causal convolution before it and gradient clipping: the C
entry points under their own names, and ``SelectiveScan`` / ``CausalConv`` /
``GradClip``, which allocate with torch, check every tensor (the library sees only
pointers) and call them.  ``include/rnn.h`` has the definitions."""
from __future__ import annotations

import array
import ctypes

from . import (RNN_BF16, RNN_F32, RNN_GATE_NONE, RNN_GATE_SILU, RNN_OK, RnnError, _p, _P, lib, rnn_conv_desc_t,
               rnn_conv_in_t, rnn_scan_desc_t, rnn_scan_grad_t, rnn_scan_in_t)
from .lm import _Op


# --- the C entry points, same names -----------------------------------------
def rnn_scan_create(desc: rnn_scan_desc_t) -> int:
    h = _P()
    rc = lib().rnn_scan_create(ctypes.byref(desc), ctypes.byref(h))
    if rc != RNN_OK:
        raise RnnError(rc, "rnn_scan_create")
    return h.value


def rnn_scan_destroy(handle: int) -> None:
    lib().rnn_scan_destroy(handle)


def rnn_scan_get_sizes(handle: int):
    """(workspace, backward workspace, reserve) bytes."""
    v = [ctypes.c_size_t() for _ in range(3)]
    rc = lib().rnn_scan_get_sizes(handle, *(ctypes.byref(x) for x in v))
    if rc != RNN_OK:
        raise RnnError(rc, "rnn_scan_get_sizes")
    return tuple(x.value for x in v)


def _set_lengths(fn, handle, lengths) -> int:
    if lengths is None:
        return fn(handle, None)
    return fn(handle, (ctypes.c_int * len(lengths))(*[int(v) for v in lengths]))


def rnn_scan_set_seq_lengths(handle, lengths) -> int:
    """lengths: a sequence of batch ints in [0, seq_len], or None for full length."""
    return _set_lengths(lib().rnn_scan_set_seq_lengths, handle, lengths)


def rnn_scan_forward(handle, inputs: rnn_scan_in_t, h0, y, hT, workspace, reserve, stream=None) -> int:
    return lib().rnn_scan_forward(handle, ctypes.byref(inputs), h0, y, hT, workspace, reserve, stream)


def rnn_scan_backward(handle, inputs: rnn_scan_in_t, dy, dhT, grad: rnn_scan_grad_t, workspace, reserve, stream=None) -> int:
    return lib().rnn_scan_backward(handle, ctypes.byref(inputs), dy, dhT, ctypes.byref(grad), workspace, reserve, stream)


def rnn_scan_step(handle, inputs: rnn_scan_in_t, state, num_slots, slots, y, stream=None) -> int:
    return lib().rnn_scan_step(handle, ctypes.byref(inputs), state, num_slots, slots, y, stream)


def rnn_scan_launch_count(handle) -> int:
    return int(lib().rnn_scan_launch_count(handle))


def rnn_conv_create(desc: rnn_conv_desc_t) -> int:
    h = _P()
    rc = lib().rnn_conv_create(ctypes.byref(desc), ctypes.byref(h))
    if rc != RNN_OK:
        raise RnnError(rc, "rnn_conv_create")
    return h.value


def rnn_conv_destroy(handle: int) -> None:
    lib().rnn_conv_destroy(handle)


def rnn_conv_get_sizes(handle: int) -> int:
    v = ctypes.c_size_t()
    rc = lib().rnn_conv_get_sizes(handle, ctypes.byref(v))
    if rc != RNN_OK:
        raise RnnError(rc, "rnn_conv_get_sizes")
    return v.value


def rnn_conv_set_seq_lengths(handle, lengths) -> int:
    """lengths: a sequence of batch ints in [0, seq_len], or None for full length."""
    return _set_lengths(lib().rnn_conv_set_seq_lengths, handle, lengths)


def rnn_conv_forward(handle, inputs: rnn_conv_in_t, s0, y, sT, stream=None) -> int:
    return lib().rnn_conv_forward(handle, ctypes.byref(inputs), s0, y, sT, stream)


def rnn_conv_backward(handle, inputs: rnn_conv_in_t, s0, dy, dsT, dx, dw, dbias, ds0, workspace, stream=None) -> int:
    return lib().rnn_conv_backward(handle, ctypes.byref(inputs), s0, dy, dsT, dx, dw, dbias, ds0, workspace, stream)


def rnn_conv_step(handle, inputs: rnn_conv_in_t, state, num_slots, slots, y, stream=None) -> int:
    return lib().rnn_conv_step(handle, ctypes.byref(inputs), state, num_slots, slots, y, stream)


def rnn_conv_launch_count(handle) -> int:
    return int(lib().rnn_conv_launch_count(handle))


def rnn_clip_create(counts, dtypes) -> int:
    """counts: elements of each tensor; dtypes: RNN_F32 or RNN_BF16 of each."""
    n = len(counts)
    h = _P()
    rc = lib().rnn_clip_create(n, (ctypes.c_int64 * n)(*counts), (ctypes.c_int * n)(*dtypes), ctypes.byref(h))
    if rc != RNN_OK:
        raise RnnError(rc, "rnn_clip_create")
    return h.value


def rnn_clip_destroy(handle: int) -> None:
    lib().rnn_clip_destroy(handle)


def rnn_clip_get_sizes(handle: int) -> int:
    v = ctypes.c_size_t()
    rc = lib().rnn_clip_get_sizes(handle, ctypes.byref(v))
    if rc != RNN_OK:
        raise RnnError(rc, "rnn_clip_get_sizes")
    return v.value


def _pointers(ptrs):
    """A host array of the pointers (None stands for NULL)."""
    return None if ptrs is None else array.array("Q", [p or 0 for p in ptrs])


def _address(a):
    return None if a is None else a.buffer_info()[0]


def rnn_clip_scale(handle, grads, out, max_norm, eps, norm, workspace, stream=None) -> int:
    """grads, out: device pointers of each tensor (out may be None)."""
    g, o = _pointers(grads), _pointers(out)
    return lib().rnn_clip_scale(handle, _address(g), _address(o), max_norm, eps, norm, workspace, stream)


def rnn_clip_norm(handle, grads, norm, workspace, stream=None) -> int:
    g = _pointers(grads)
    return lib().rnn_clip_norm(handle, _address(g), norm, workspace, stream)


def rnn_clip_launch_count(handle) -> int:
    return int(lib().rnn_clip_launch_count(handle))


# --- convenience wrappers (torch allocation + the calls above) ----------------
class _Sequences(_Op):
    """What the scan and the convolution share: lengths, outputs and pools of states."""

    def set_seq_lengths(self, lengths):
        """Valid tokens per sequence (batch ints), or None for full length, for the calls made from now on; waits for the
        calls before that have lengths of their own."""
        if lengths is not None and len(lengths) != self.desc.batch:
            raise ValueError("one length per sequence of the batch")
        self._check(self._lengths(self.handle, lengths), self._lengths.__name__)

    def _out(self, t, name, like):
        """The output ``t``, or a new one of the shape and dtype of the input ``like``."""
        if t is None:
            return self._dense_like(like)
        self._want(t, name, like.shape)
        return t

    def _state(self, t, name, dtype):
        if t is None:
            return self.torch.empty(self._s, dtype=dtype, device=self.device)
        self._want(t, name, self._s, dtype)
        return t

    def _pool(self, state, slots, shape, dtype):
        """The number of slots of a pool [num_slots, *shape]."""
        torch = self.torch
        if not isinstance(state, torch.Tensor) or state.dim() != 3:
            raise ValueError(f"state must be a [num_slots, {shape[0]}, {shape[1]}] tensor")
        n = state.shape[0]
        self._want(state, "state", (n,) + shape, dtype)
        if slots is None:
            if n < self.desc.batch:
                raise ValueError(f"state has {n} slots for {self.desc.batch} sequences")
        else:
            self._like(slots, "slots", (self.desc.batch,), torch.int32)
            if not slots.is_contiguous():
                raise ValueError("slots must be contiguous")
        return n


class SelectiveScan(_Sequences):
    """The selective scan over [T, B, channels] sequences ([B, T, channels] with batch_first), bound to a device.

    x, dt and z are [T, B, channels], B and C [T, B, groups, states], all in the dtype of the handle and each possibly a
    slice of a packed projection (rows of any one stride); A is fp32 [channels, states], D and dt_bias fp32 [channels],
    states fp32 [B, channels, states], all dense.  z, D and dt_bias may be left out.  Calls run on the current stream,
    or on ``stream``."""

    _destroy, _lengths = staticmethod(rnn_scan_destroy), staticmethod(rnn_scan_set_seq_lengths)

    def __init__(self, batch: int, seq_len: int, channels: int, states: int, groups: int = 1, dtype: str = "bf16",
                 softplus: bool = True, batch_first: bool = False, device=None):
        self._bind(dtype, device)
        d = rnn_scan_desc_t(batch, seq_len, channels, states, groups, RNN_BF16 if dtype == "bf16" else RNN_F32,
                            int(bool(batch_first)), int(bool(softplus)))
        self.desc = d
        with self.torch.cuda.device(self.device):
            self.handle = rnn_scan_create(d)
        self.workspace_bytes, self.backward_workspace_bytes, self.reserve_bytes = rnn_scan_get_sizes(self.handle)
        self._shapes()

    def _shapes(self):
        d = self.desc
        lead = (d.batch, d.seq_len) if d.batch_first else (d.seq_len, d.batch)
        self._x, self._bc = lead + (d.channels,), lead + (d.groups, d.states)
        self._a, self._d, self._s = (d.channels, d.states), (d.channels,), (d.batch, d.channels, d.states)

    def launches(self) -> int:
        return rnn_scan_launch_count(self.handle)

    def _inputs(self, x, dt, A, B, C, z, D, dt_bias) -> rnn_scan_in_t:
        f32 = self.torch.float32
        for t, name in ((x, "x"), (dt, "dt"), (A, "A"), (B, "B"), (C, "C")):
            if t is None:
                raise ValueError(f"{name} is required")
        self._want(A, "A", self._a, f32)
        self._want(D, "D", self._d, f32)
        self._want(dt_bias, "dt_bias", self._d, f32)
        rows = (self._rows(x, "x", self._x, 2, True), self._rows(dt, "dt", self._x, 2, True),
                0 if z is None else self._rows(z, "z", self._x, 2, True),
                self._rows(B, "B", self._bc, 2, False), self._rows(C, "C", self._bc, 2, False))
        return rnn_scan_in_t(x.data_ptr(), dt.data_ptr(), _p(z), B.data_ptr(), C.data_ptr(), A.data_ptr(), _p(D),
                             _p(dt_bias), *rows)

    def forward(self, x, dt, A, B, C, z=None, D=None, dt_bias=None, h0=None, train=True, y=None, hT=None, stream=None):
        """(y, hT).  ``train`` keeps what backward needs until the next training forward.  hT may be h0."""
        if stream is not None:
            return self._elsewhere(self.forward, stream, x, dt, A, B, C, z=z, D=D, dt_bias=dt_bias, h0=h0, train=train,
                                   y=y, hT=hT)
        f32 = self.torch.float32
        a = self._inputs(x, dt, A, B, C, z, D, dt_bias)
        self._want(h0, "h0", self._s, f32)
        y, hT = self._out(y, "y", x), self._state(hT, "hT", f32)
        raw = self._on()
        ws = self._scratch("workspace", self.workspace_bytes, raw) if self.workspace_bytes else None
        rs = self._scratch("reserve", self.reserve_bytes, raw) if train else None
        rc = rnn_scan_forward(self.handle, a, _p(h0), y.data_ptr(), hT.data_ptr(), _p(ws), _p(rs), raw)
        self._check(rc, "rnn_scan_forward")
        return y, hT

    def backward(self, dy, x, dt, A, B, C, z=None, D=None, dt_bias=None, dhT=None, stream=None):
        """A dict of the gradients dx, ddt, dz, dB, dC (handle's dtype), dA, dD, ddt_bias and dh0 (fp32) after a training
        forward of the same inputs; None where the call leaves the input out."""
        if stream is not None:
            return self._elsewhere(self.backward, stream, dy, x, dt, A, B, C, z=z, D=D, dt_bias=dt_bias, dhT=dhT)
        f32 = self.torch.float32
        if getattr(self, "reserve", None) is None:
            raise ValueError("backward needs a training forward first")
        if dy is None:
            raise ValueError("dy is required")
        a = self._inputs(x, dt, A, B, C, z, D, dt_bias)
        self._want(dy, "dy", self._x)
        self._want(dhT, "dhT", self._s, f32)
        new = self._dense_like
        out = {"dx": new(x), "ddt": new(x), "dz": None if z is None else new(x), "dB": new(B), "dC": new(B), "dA": new(A),
               "dD": None if D is None else new(D), "ddt_bias": None if dt_bias is None else new(dt_bias),
               "dh0": self._state(None, "dh0", f32)}
        raw = self._on()
        ws = self._scratch("backward_workspace", self.backward_workspace_bytes, raw)
        rs = self._scratch("reserve", self.reserve_bytes, raw)
        rc = rnn_scan_backward(self.handle, a, dy.data_ptr(), _p(dhT), rnn_scan_grad_t(*(_p(t) for t in out.values())),
                               _p(ws), _p(rs), raw)
        self._check(rc, "rnn_scan_backward")
        return out

    def step(self, x, dt, A, B, C, state, z=None, D=None, dt_bias=None, slots=None, y=None, stream=None):
        """seq_len new tokens of each sequence against ``state`` [num_slots, channels, states] fp32, updated in place;
        ``slots`` int32 [batch] names each sequence's state (a slot outside the pool skips the sequence)."""
        if stream is not None:
            return self._elsewhere(self.step, stream, x, dt, A, B, C, state, z=z, D=D, dt_bias=dt_bias, slots=slots, y=y)
        a = self._inputs(x, dt, A, B, C, z, D, dt_bias)
        n = self._pool(state, slots, self._a, self.torch.float32)
        y = self._out(y, "y", x)
        rc = rnn_scan_step(self.handle, a, state.data_ptr(), n, _p(slots), y.data_ptr(), self._on())
        self._check(rc, "rnn_scan_step")
        return y


class CausalConv(_Sequences):
    """The depthwise causal convolution over [T, B, channels] sequences ([B, T, channels] with batch_first), bound to a
    device.

    x may be a slice of a packed projection (rows of any one stride); w is [channels, width], bias [channels] or left
    out, states [B, width - 1, channels], oldest input first; everything in the dtype of the handle, and dense but x.
    ``act`` is None or "silu".  Calls run on the current stream, or on ``stream``."""

    _destroy, _lengths = staticmethod(rnn_conv_destroy), staticmethod(rnn_conv_set_seq_lengths)
    _acts = {None: RNN_GATE_NONE, "silu": RNN_GATE_SILU}

    def __init__(self, batch: int, seq_len: int, channels: int, width: int = 4, dtype: str = "bf16", act="silu",
                 batch_first: bool = False, device=None):
        if act not in self._acts:
            raise ValueError(f"act must be None or 'silu', not {act!r}")
        self._bind(dtype, device)
        d = rnn_conv_desc_t(batch, seq_len, channels, width, RNN_BF16 if dtype == "bf16" else RNN_F32,
                            int(bool(batch_first)), self._acts[act])
        self.desc = d
        with self.torch.cuda.device(self.device):
            self.handle = rnn_conv_create(d)
        self.backward_workspace_bytes = rnn_conv_get_sizes(self.handle)
        self._shapes()

    def _shapes(self):
        d = self.desc
        self._x = ((d.batch, d.seq_len) if d.batch_first else (d.seq_len, d.batch)) + (d.channels,)
        self._w, self._b, self._s = (d.channels, d.width), (d.channels,), (d.batch, d.width - 1, d.channels)

    def launches(self) -> int:
        return rnn_conv_launch_count(self.handle)

    def _inputs(self, x, w, bias) -> rnn_conv_in_t:
        for t, name in ((x, "x"), (w, "w")):
            if t is None:
                raise ValueError(f"{name} is required")
        self._want(w, "w", self._w)
        self._want(bias, "bias", self._b)
        return rnn_conv_in_t(x.data_ptr(), w.data_ptr(), _p(bias), self._rows(x, "x", self._x, 2, True))

    def forward(self, x, w, bias=None, s0=None, y=None, sT=None, stream=None):
        """(y, sT).  sT may be s0; y lies apart from x."""
        if stream is not None:
            return self._elsewhere(self.forward, stream, x, w, bias=bias, s0=s0, y=y, sT=sT)
        a = self._inputs(x, w, bias)
        self._want(s0, "s0", self._s)
        y, sT = self._out(y, "y", x), self._state(sT, "sT", self.tdtype)
        rc = rnn_conv_forward(self.handle, a, _p(s0), y.data_ptr(), sT.data_ptr(), self._on())
        self._check(rc, "rnn_conv_forward")
        return y, sT

    def backward(self, dy, x, w, bias=None, s0=None, dsT=None, stream=None):
        """A dict of the gradients dx, ds0 (handle's dtype), dw and dbias (fp32; None without a bias) of a forward call
        with these inputs."""
        if stream is not None:
            return self._elsewhere(self.backward, stream, dy, x, w, bias=bias, s0=s0, dsT=dsT)
        f32 = self.torch.float32
        if dy is None:
            raise ValueError("dy is required")
        a = self._inputs(x, w, bias)
        self._want(dy, "dy", self._x)
        self._want(s0, "s0", self._s)
        self._want(dsT, "dsT", self._s)
        torch = self.torch
        out = {"dx": self._dense_like(x), "dw": torch.empty_like(w, dtype=f32),
               "dbias": None if bias is None else torch.empty_like(bias, dtype=f32), "ds0": self._state(None, "ds0", self.tdtype)}
        raw = self._on()
        ws = self._scratch("backward_workspace", self.backward_workspace_bytes, raw)
        rc = rnn_conv_backward(self.handle, a, _p(s0), dy.data_ptr(), _p(dsT), *(_p(t) for t in out.values()), _p(ws), raw)
        self._check(rc, "rnn_conv_backward")
        return out

    def step(self, x, w, state, bias=None, slots=None, y=None, stream=None):
        """seq_len new tokens of each sequence against ``state`` [num_slots, width - 1, channels], updated in place;
        ``slots`` as in SelectiveScan.step."""
        if stream is not None:
            return self._elsewhere(self.step, stream, x, w, state, bias=bias, slots=slots, y=y)
        a = self._inputs(x, w, bias)
        n = self._pool(state, slots, self._s[1:], self.tdtype)
        y = self._out(y, "y", x)
        rc = rnn_conv_step(self.handle, a, state.data_ptr(), n, _p(slots), y.data_ptr(), self._on())
        self._check(rc, "rnn_conv_step")
        return y


class GradClip(_Op):
    """The norm of a list of gradients together, and their scaling where it is over a limit, bound to a device.

    ``counts`` are the elements of each tensor, ``dtypes`` "f32" or "bf16" for all of them or one for each.  Tensors are
    contiguous, of any shape and alignment (slices of a flat gradient among them), in a list or anything that can be
    gone through (``dict.values()``)."""

    _destroy = staticmethod(rnn_clip_destroy)

    def __init__(self, counts, dtypes="f32", device=None):
        counts = [int(n) for n in counts]
        dtypes = [dtypes] * len(counts) if isinstance(dtypes, str) else list(dtypes)
        if len(dtypes) != len(counts):
            raise ValueError("one dtype per tensor, or one for all")
        for d in dtypes:
            if d not in ("bf16", "f32"):
                raise ValueError(f"dtypes must be 'bf16' or 'f32', not {d!r}")
        self._bind("f32", device)
        torch = self.torch
        self.desc = list(zip(counts, (torch.bfloat16 if d == "bf16" else torch.float32 for d in dtypes)))
        self._counts, self._dtypes = counts, [dt for _, dt in self.desc]
        with torch.cuda.device(self.device):
            self.handle = rnn_clip_create(counts, [RNN_BF16 if d == "bf16" else RNN_F32 for d in dtypes])
        self.workspace_bytes = rnn_clip_get_sizes(self.handle)

    def launches(self) -> int:
        return rnn_clip_launch_count(self.handle)

    @staticmethod
    def _listed(tensors):
        """A dict's values or a generator as a list: it is gone through more than once, and a call on another stream
        has to name each tensor to the allocator."""
        return tensors if isinstance(tensors, (list, tuple)) else list(tensors)

    def _tensors(self, tensors, name):
        """The pointers of a list of tensors that are as the handle has them."""
        if len(tensors) != len(self.desc):
            raise ValueError(f"{name} has {len(tensors)} tensors; the handle has {len(self.desc)}")
        # one pass over what is usually right; what is wrong is found again below
        torch, n = self.torch, len(tensors)
        T = torch.Tensor
        try:
            if (list(map(T.numel, tensors)) == self._counts and list(map(T.get_device, tensors)) == [self.device.index] * n
                    and [t.dtype for t in tensors] == self._dtypes and all(map(T.is_contiguous, tensors))):
                return list(map(T.data_ptr, tensors))
        except TypeError:
            pass
        for i, (t, (n, dt)) in enumerate(zip(tensors, self.desc)):
            if not isinstance(t, T):
                raise TypeError(f"{name}[{i}] must be a torch.Tensor, not {type(t).__name__}")
            if t.device != self.device:
                raise ValueError(f"{name}[{i}] is on {t.device}; the handle is on {self.device}")
            if t.dtype != dt or t.numel() != n:
                raise ValueError(f"{name}[{i}] has {t.numel()} elements of {t.dtype}; expected {n} of {dt}")
            if not t.is_contiguous():
                raise ValueError(f"{name}[{i}] must be contiguous")
        raise ValueError(f"{name}: not as the handle has it")

    def _norm(self, norm):
        if norm is None:
            return self.torch.empty(1, dtype=self.torch.float32, device=self.device)
        self._like(norm, "norm", (1,), self.torch.float32)
        return norm

    def clip(self, grads, max_norm: float, eps: float = 1e-6, out=None, norm=None, stream=None):
        """Scales ``grads`` by min(1, max_norm / (norm + eps)), in place or into the tensors of ``out`` (each its gradient,
        or memory that no gradient shares; nothing is written twice), and returns the norm before it (fp32 [1] on the
        device; infinity where fp32 cannot hold it).  With a NaN or infinity among them the values stay as they are."""
        grads, out = self._listed(grads), None if out is None else self._listed(out)
        if stream is not None:
            return self._elsewhere(self.clip, stream, grads, max_norm, eps=eps, out=out, norm=norm)
        p = self._tensors(grads, "grads")
        q = None if out is None else self._tensors(out, "out")
        norm = self._norm(norm)
        raw = self._on()
        ws = self._scratch("workspace", self.workspace_bytes, raw)
        rc = rnn_clip_scale(self.handle, p, q, max_norm, eps, norm.data_ptr(), ws.data_ptr(), raw)
        self._check(rc, "rnn_clip_scale")
        return norm

    def norm(self, grads, norm=None, stream=None):
        """The norm of ``grads`` together (fp32 [1] on the device)."""
        grads = self._listed(grads)
        if stream is not None:
            return self._elsewhere(self.norm, stream, grads, norm=norm)
        p = self._tensors(grads, "grads")
        norm = self._norm(norm)
        raw = self._on()
        ws = self._scratch("workspace", self.workspace_bytes, raw)
        rc = rnn_clip_norm(self.handle, p, norm.data_ptr(), ws.data_ptr(), raw)
        self._check(rc, "rnn_clip_norm")
        return norm
