"""The gated delta rule and the block norm: the C entry points under their own
names, and ``DeltaRule`` / ``BlockNorm``, which allocate with torch, check every
tensor (the library sees only pointers) and call them.  ``include/rnn.h`` has
the definitions."""
from __future__ import annotations

import ctypes
import math

from . import (RNN_BF16, RNN_F32, RNN_GATE_NONE, RNN_GATE_SIGMOID, RNN_GATE_SILU, RNN_OK, RnnError, _p, _P, lib,
                rnn_delta_desc_t, rnn_delta_in_t, rnn_norm_desc_t, rnn_norm_in_t)


# --- the C entry points, same names -----------------------------------------
def rnn_delta_create(desc: rnn_delta_desc_t) -> int:
    h = _P()
    rc = lib().rnn_delta_create(ctypes.byref(desc), ctypes.byref(h))
    if rc != RNN_OK:
        raise RnnError(rc, "rnn_delta_create")
    return h.value


def rnn_delta_destroy(handle: int) -> None:
    lib().rnn_delta_destroy(handle)


def rnn_delta_get_sizes(handle: int):
    """(workspace, backward workspace, reserve) bytes."""
    v = [ctypes.c_size_t() for _ in range(3)]
    rc = lib().rnn_delta_get_sizes(handle, *(ctypes.byref(x) for x in v))
    if rc != RNN_OK:
        raise RnnError(rc, "rnn_delta_get_sizes")
    return tuple(x.value for x in v)


def rnn_delta_set_seq_lengths(handle, lengths) -> int:
    """lengths: a sequence of batch ints in [0, seq_len], or None for full length."""
    if lengths is None:
        return lib().rnn_delta_set_seq_lengths(handle, None)
    arr = (ctypes.c_int * len(lengths))(*[int(v) for v in lengths])
    return lib().rnn_delta_set_seq_lengths(handle, arr)


def rnn_delta_forward(handle, inputs: rnn_delta_in_t, s0, o, sT, workspace, reserve, stream=None) -> int:
    return lib().rnn_delta_forward(handle, ctypes.byref(inputs), s0, o, sT, workspace, reserve, stream)


def rnn_delta_backward(handle, inputs: rnn_delta_in_t, do, dsT, dq, dk, dv, dg, dbeta, ds0, workspace, reserve,
                       stream=None) -> int:
    return lib().rnn_delta_backward(handle, ctypes.byref(inputs), do, dsT, dq, dk, dv, dg, dbeta, ds0, workspace,
                                    reserve, stream)


def rnn_delta_step(handle, inputs: rnn_delta_in_t, state, num_slots, slots, o, stream=None) -> int:
    return lib().rnn_delta_step(handle, ctypes.byref(inputs), state, num_slots, slots, o, stream)


def rnn_delta_sync_status(handle, stream=None) -> int:
    return lib().rnn_delta_sync_status(handle, stream)


def rnn_delta_launch_count(handle) -> int:
    return int(lib().rnn_delta_launch_count(handle))


def rnn_norm_create(desc: rnn_norm_desc_t) -> int:
    h = _P()
    rc = lib().rnn_norm_create(ctypes.byref(desc), ctypes.byref(h))
    if rc != RNN_OK:
        raise RnnError(rc, "rnn_norm_create")
    return h.value


def rnn_norm_destroy(handle: int) -> None:
    lib().rnn_norm_destroy(handle)


def rnn_norm_get_sizes(handle: int) -> int:
    v = ctypes.c_size_t()
    rc = lib().rnn_norm_get_sizes(handle, ctypes.byref(v))
    if rc != RNN_OK:
        raise RnnError(rc, "rnn_norm_get_sizes")
    return v.value


def rnn_norm_forward(handle, inputs: rnn_norm_in_t, x_out, n_out, stream=None) -> int:
    return lib().rnn_norm_forward(handle, ctypes.byref(inputs), x_out, n_out, stream)


def rnn_norm_backward(handle, inputs: rnn_norm_in_t, dx_out, dn_out, dy, dz, dx, dw_in, dscale, dw_out, workspace,
                      stream=None) -> int:
    return lib().rnn_norm_backward(handle, ctypes.byref(inputs), dx_out, dn_out, dy, dz, dx, dw_in, dscale, dw_out,
                                   workspace, stream)


def rnn_norm_launch_count(handle) -> int:
    return int(lib().rnn_norm_launch_count(handle))


# --- convenience wrappers (torch allocation + the calls above) ----------------
class _Op:
    """What the two wrappers share: the device, the handle's life and the tensor checks."""

    def _bind(self, dtype: str, device):
        if dtype not in ("bf16", "f32"):
            raise ValueError(f"dtype must be 'bf16' or 'f32', not {dtype!r}")
        import torch
        self.torch = torch
        self.tdtype = torch.bfloat16 if dtype == "bf16" else torch.float32
        self._users = {}          # of each scratch buffer: raw streams
        self.device = torch.device(device if device is not None else "cuda")
        if self.device.index is None:     # pin the device current now: the handle is bound to it
            self.device = torch.device("cuda", torch.cuda.current_device())

    def close(self):
        if getattr(self, "handle", None):
            self._destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _scratch(self, name: str, nbytes: int, raw: int):
        """The scratch buffer ``name``, allocated at its first use, for a call on the current stream (``raw``).  The
        library orders the calls that share it; the allocator learns of every stream that uses it."""
        t = getattr(self, name, None)
        if t is None:
            t = self.torch.empty(max(nbytes, 256), dtype=self.torch.uint8, device=self.device)
            setattr(self, name, t)
            self._users[name] = {raw}
        elif raw not in self._users[name]:
            self._users[name].add(raw)
            t.record_stream(self.torch.cuda.current_stream(self.device))
        return t

    def _want(self, t, name: str, shape, dtype=None):
        """Raise unless ``t`` (None passes) is a contiguous, 16-byte aligned tensor of this shape and dtype on the
        handle's device."""
        if t is None:
            return
        self._like(t, name, shape, dtype)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.data_ptr() & 15:
            raise ValueError(f"{name} must start on a 16-byte boundary")

    def _like(self, t, name: str, shape, dtype=None):
        # one pass over what is usually right; what is wrong is found again below
        try:
            if t.dtype is (dtype or self.tdtype) and t.shape == shape and t.device == self.device:
                return
        except AttributeError:
            pass
        if not isinstance(t, self.torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor, not {type(t).__name__}")
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}; the handle is on {self.device}")
        if t.dtype != (dtype or self.tdtype):
            raise ValueError(f"{name} has dtype {t.dtype}; expected {dtype or self.tdtype}")
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {tuple(shape)}")

    def _on(self) -> int:
        """The device's current stream (its handle alone: making the Stream object costs as much as the launch)."""
        return self.torch._C._cuda_getCurrentRawStream(self.device.index)

    def _elsewhere(self, call, stream, *tensors, **more):
        """``call`` made with ``stream`` current, for a caller whose current stream is another: what it allocates is
        that stream's own memory, and neither its tensors nor the results are reused before both streams are done with
        them.  Ordering the call after what made its inputs, and the results' use after the call, is the caller's."""
        torch = self.torch
        if stream.device != self.device:
            raise ValueError(f"stream is on {stream.device}; the handle is on {self.device}")
        here = torch.cuda.current_stream(self.device)
        with torch.cuda.stream(stream):
            out = call(*tensors, **more)
        for t in (*tensors, *more.values()):
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)
        results = (out,) if isinstance(out, torch.Tensor) else out.values() if isinstance(out, dict) else out
        for t in results:
            if t is not None:
                t.record_stream(here)
        return out

    def _rows(self, t, name: str, shape, lead: int, align: bool) -> int:
        """Row stride (elements) of ``t``: its first ``lead`` dimensions run over rows of one stride, the others are
        dense."""
        self._like(t, name, shape)
        dense = math.prod(shape[lead:])
        if t.is_contiguous():
            row = dense
        else:
            st = t.stride()
            row = st[lead - 1]
            inner = st[-1] == 1 and (len(shape) == lead + 1 or st[lead] == shape[-1])
            if not (inner and row >= dense and (lead == 1 or st[0] == shape[1] * row)):
                row = self._slow_rows(st, name, shape, lead, dense)
        if align and (t.data_ptr() & 15 or (row * t.element_size()) & 15):
            raise ValueError(f"{name}: rows must start on 16-byte boundaries")
        return row

    @staticmethod
    def _slow_rows(st, name, shape, lead, dense):
        """_rows where dimensions of one element carry any stride, or where something is wrong."""
        size = 1
        for n, s in zip(reversed(shape[lead:]), reversed(st[lead:])):
            if n > 1 and s != size:
                raise ValueError(f"{name}: the elements of a row must be contiguous")
            size *= n
        row, want = dense, None
        for n, s in zip(reversed(shape[:lead]), reversed(st[:lead])):
            if n > 1:
                if want is None:
                    row = s
                elif s != want:
                    raise ValueError(f"{name}: consecutive rows must have one stride")
                want = n * s
        if row < dense:
            raise ValueError(f"{name}: rows must not overlap")
        return row

    def _dense_like(self, t):
        """A new dense tensor of ``t``'s shape and dtype."""
        return self.torch.empty_like(t, memory_format=self.torch.contiguous_format)

    def _check(self, rc, what):
        if rc != RNN_OK:
            raise RnnError(rc, what)


class DeltaRule(_Op):
    """The gated delta rule over [T, B, heads, dim] sequences ([B, T, heads, dim] with batch_first), bound to a device.

    q and k have ``heads_k`` heads of ``dim_k``, v and o ``heads_v`` heads of ``dim_v``, g (log decay) and beta
    [T, B, heads_v]; all in the dtype of the handle, the states fp32 [B, heads_v, dim_v, dim_k].  q, k, v, g and beta may
    be slices of packed projections (rows of any one stride); every other tensor is dense.  Calls run on the current
    stream, or on ``stream``."""

    _destroy = staticmethod(rnn_delta_destroy)

    def __init__(self, batch: int, seq_len: int, heads_k: int, heads_v: int, dim_k: int, dim_v: int,
                 dtype: str = "bf16", scale: float = 0.0, batch_first: bool = False, device=None):
        self._bind(dtype, device)
        d = rnn_delta_desc_t(batch, seq_len, heads_k, heads_v, dim_k, dim_v,
                             RNN_BF16 if dtype == "bf16" else RNN_F32, int(bool(batch_first)), float(scale))
        self.desc = d
        with self.torch.cuda.device(self.device):
            self.handle = rnn_delta_create(d)
        self.workspace_bytes, self.backward_workspace_bytes, self.reserve_bytes = rnn_delta_get_sizes(self.handle)
        self._shapes()

    def _shapes(self):
        d = self.desc
        lead = (d.batch, d.seq_len) if d.batch_first else (d.seq_len, d.batch)
        self._qk, self._v, self._g = lead + (d.heads_k, d.dim_k), lead + (d.heads_v, d.dim_v), lead + (d.heads_v,)
        self._s = (d.batch, d.heads_v, d.dim_v, d.dim_k)

    def launches(self) -> int:
        return rnn_delta_launch_count(self.handle)

    def sync(self, stream=None):
        """Wait for the stream and raise what a kernel reported."""
        raw = self._on() if stream is None else stream.cuda_stream
        self._check(rnn_delta_sync_status(self.handle, raw), "rnn_delta_sync_status")

    def set_seq_lengths(self, lengths):
        """Valid tokens per sequence (batch ints), or None for full length, for the calls made from now on; waits for the
        calls before that have lengths of their own."""
        if lengths is not None and len(lengths) != self.desc.batch:
            raise ValueError("one length per sequence of the batch")
        self._check(rnn_delta_set_seq_lengths(self.handle, lengths), "rnn_delta_set_seq_lengths")

    def _inputs(self, q, k, v, g, beta) -> rnn_delta_in_t:
        rows = (self._rows(q, "q", self._qk, 2, True), self._rows(k, "k", self._qk, 2, True),
                self._rows(v, "v", self._v, 2, True), self._rows(g, "g", self._g, 2, False),
                self._rows(beta, "beta", self._g, 2, False))
        return rnn_delta_in_t(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), *rows)

    def _out(self, t, name, shape, like):
        if t is None:
            return self._dense_like(like)
        self._want(t, name, shape)
        return t

    def _state(self, t, name):
        if t is None:
            return self.torch.empty(self._s, dtype=self.torch.float32, device=self.device)
        self._want(t, name, self._s, self.torch.float32)
        return t

    def forward(self, q, k, v, g, beta, s0=None, train=True, o=None, sT=None, stream=None):
        """(o, sT).  ``train`` keeps what backward needs until the next training forward."""
        if stream is not None:
            return self._elsewhere(self.forward, stream, q, k, v, g, beta, s0=s0, train=train, o=o, sT=sT)
        f32 = self.torch.float32
        x = self._inputs(q, k, v, g, beta)
        self._want(s0, "s0", self._s, f32)
        o, sT = self._out(o, "o", self._v, v), self._state(sT, "sT")
        raw = self._on()
        ws = self._scratch("workspace", self.workspace_bytes, raw)
        rs = self._scratch("reserve", self.reserve_bytes, raw) if train else None
        rc = rnn_delta_forward(self.handle, x, _p(s0), _p(o), _p(sT), _p(ws), _p(rs), raw)
        self._check(rc, "rnn_delta_forward")
        return o, sT

    def backward(self, do, q, k, v, g, beta, s0=None, dsT=None, ds0=None, stream=None):
        """(dq, dk, dv, dg, dbeta, ds0) after a training forward of the same inputs.  s0 is accepted for symmetry: what
        backward needs of it is in the reserve."""
        if stream is not None:
            return self._elsewhere(self.backward, stream, do, q, k, v, g, beta, s0=s0, dsT=dsT, ds0=ds0)
        f32 = self.torch.float32
        if getattr(self, "reserve", None) is None:
            raise ValueError("backward needs a training forward first")
        x = self._inputs(q, k, v, g, beta)
        if do is None:
            raise ValueError("do is required")
        self._want(do, "do", self._v)
        self._want(dsT, "dsT", self._s, f32)
        dq, dk, dv, dg, dbeta = (self._dense_like(t) for t in (q, k, v, g, beta))
        ds0 = self._state(ds0, "ds0")
        raw = self._on()
        ws = self._scratch("backward_workspace", self.backward_workspace_bytes, raw)
        rs = self._scratch("reserve", self.reserve_bytes, raw)
        rc = rnn_delta_backward(self.handle, x, _p(do), _p(dsT), _p(dq), _p(dk), _p(dv), _p(dg), _p(dbeta), _p(ds0),
                                _p(ws), _p(rs), raw)
        self._check(rc, "rnn_delta_backward")
        return dq, dk, dv, dg, dbeta, ds0

    def step(self, q, k, v, g, beta, state, slots=None, o=None, stream=None):
        """seq_len new tokens of each sequence against ``state`` [num_slots, heads_v, dim_v, dim_k] fp32, updated in
        place; ``slots`` int32 [batch] names each sequence's state (a slot outside the pool skips the sequence)."""
        if stream is not None:
            return self._elsewhere(self.step, stream, q, k, v, g, beta, state, slots=slots, o=o)
        torch, d = self.torch, self.desc
        x = self._inputs(q, k, v, g, beta)
        if not isinstance(state, torch.Tensor) or state.dim() != 4:
            raise ValueError("state must be a [num_slots, heads_v, dim_v, dim_k] tensor")
        n = state.shape[0]
        self._want(state, "state", (n,) + self._s[1:], torch.float32)
        if slots is None:
            if n < d.batch:
                raise ValueError(f"state has {n} slots for {d.batch} sequences")
        else:
            self._like(slots, "slots", (d.batch,), torch.int32)
            if not slots.is_contiguous():
                raise ValueError("slots must be contiguous")
        o = self._out(o, "o", self._v, v)
        rc = rnn_delta_step(self.handle, x, state.data_ptr(), n, _p(slots), o.data_ptr(), self._on())
        self._check(rc, "rnn_delta_step")
        return o


class BlockNorm(_Op):
    """The norms, gate and scaled residual around a block, over [rows, groups * cols] tensors:

        b = RMSNorm(y; w_in) * act(z),  x' = x + scale * b,  n = RMSNorm(x'; w_out)

    with any of the parts left out.  y, z and x may be slices of wider rows; weights are [cols] of the handle's dtype,
    None standing for ones."""

    _destroy = staticmethod(rnn_norm_destroy)
    _gates = {None: RNN_GATE_NONE, "silu": RNN_GATE_SILU, "sigmoid": RNN_GATE_SIGMOID}

    def __init__(self, rows: int, cols: int, groups: int = 1, dtype: str = "bf16", norm_in: bool = True, gate=None,
                 residual: bool = False, norm_out: bool = False, eps: float = 1e-6, device=None):
        if gate not in self._gates:
            raise ValueError(f"gate must be None, 'silu' or 'sigmoid', not {gate!r}")
        self._bind(dtype, device)
        d = rnn_norm_desc_t(rows, groups, cols, RNN_BF16 if dtype == "bf16" else RNN_F32, int(bool(norm_in)),
                            self._gates[gate], int(bool(residual)), int(bool(norm_out)), float(eps))
        self.desc = d
        with self.torch.cuda.device(self.device):
            self.handle = rnn_norm_create(d)
        self.workspace_bytes = rnn_norm_get_sizes(self.handle)
        self._shapes()

    def _shapes(self):
        d = self.desc
        self._full, self._w = (d.rows, d.groups * d.cols), (d.cols,)

    def launches(self) -> int:
        return rnn_norm_launch_count(self.handle)

    def _inputs(self, y, z, x, w_in, scale, w_out) -> rnn_norm_in_t:
        d = self.desc
        for t, name, on in ((z, "z", d.gate), (x, "x", d.residual)):
            if bool(on) != (t is not None):
                raise ValueError(f"{name} is {'required' if on else 'not used'} by this handle")
        for t, name, on in ((w_in, "w_in", d.norm_in), (scale, "scale", d.residual), (w_out, "w_out", d.norm_out)):
            if t is not None and not on:
                raise ValueError(f"{name} is not used by this handle")
            self._want(t, name, self._w)
        r = [0 if t is None else self._rows(t, n, self._full, 1, True) for t, n in ((y, "y"), (z, "z"), (x, "x"))]
        return rnn_norm_in_t(y.data_ptr(), _p(z), _p(x), _p(w_in), _p(scale), _p(w_out), *r)

    def forward(self, y, z=None, x=None, w_in=None, scale=None, w_out=None, x_out=None, n_out=None, stream=None):
        """(x_out, n_out); n_out is None without norm_out.  x_out may be x itself."""
        if stream is not None:
            return self._elsewhere(self.forward, stream, y, z=z, x=x, w_in=w_in, scale=scale, w_out=w_out, x_out=x_out,
                                   n_out=n_out)
        if y is None:
            raise ValueError("y is required")
        a = self._inputs(y, z, x, w_in, scale, w_out)
        if x_out is None:
            x_out = self._dense_like(y)
        else:
            self._want(x_out, "x_out", self._full)
        if not self.desc.norm_out:
            if n_out is not None:
                raise ValueError("n_out is not used by this handle")
        elif n_out is None:
            n_out = self._dense_like(y)
        else:
            self._want(n_out, "n_out", self._full)
        rc = rnn_norm_forward(self.handle, a, x_out.data_ptr(), _p(n_out), self._on())
        self._check(rc, "rnn_norm_forward")
        return x_out, n_out

    def backward(self, dx_out, dn_out, y, z=None, x=None, w_in=None, scale=None, w_out=None, stream=None):
        """A dict of the gradients dy, dz, dx (handle's dtype) and dw_in, dscale, dw_out (fp32); None where the handle
        or the call leaves the input out.  dx_out or dn_out may be None."""
        if stream is not None:
            return self._elsewhere(self.backward, stream, dx_out, dn_out, y, z=z, x=x, w_in=w_in, scale=scale,
                                   w_out=w_out)
        d, torch = self.desc, self.torch
        if y is None:
            raise ValueError("y is required")
        if dx_out is None and dn_out is None:
            raise ValueError("dx_out or dn_out is required")
        if dn_out is not None and not d.norm_out:
            raise ValueError("dn_out is not used by this handle")
        a = self._inputs(y, z, x, w_in, scale, w_out)
        self._want(dx_out, "dx_out", self._full)
        self._want(dn_out, "dn_out", self._full)

        out = {"dy": self._dense_like(y), "dz": self._dense_like(y) if d.gate else None,
               "dx": self._dense_like(y) if d.residual else None}
        weights = False
        for name, t in (("dw_in", w_in), ("dscale", scale), ("dw_out", w_out)):
            out[name] = None if t is None else torch.empty_like(t, dtype=torch.float32)
            weights = weights or t is not None
        raw = self._on()
        ws = self._scratch("workspace", self.workspace_bytes, raw) if weights else None
        rc = rnn_norm_backward(self.handle, a, _p(dx_out), _p(dn_out), *(_p(t) for t in out.values()), _p(ws), raw)
        self._check(rc, "rnn_norm_backward")
        return out
