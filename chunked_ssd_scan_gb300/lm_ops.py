"""Operators around a scan in a recurrent language model: the gated linear recurrence, the
channels-last group norm with an activation and the token embedding (declarations and contracts
in include/ssdscan.h).

Every operator is a function and a plan.  A plan checks its arguments, allocates outputs and
workspace once and makes only the C call when it is called; the function makes a plan and calls it.
With ``stream`` given, what is allocated here belongs to that stream, and the memory of the inputs,
and of outputs and a workspace that the caller passes, is kept from reuse until the work on that
stream is done.

A ``workspace`` of the caller's is a uint8 tensor of at least as many bytes as the operator's
``..._workspace_bytes`` function in the C library says, on the inputs' device.  Its first
``HEADER_BYTES`` are zero before its first call (the recurrence counts its tiles there and leaves
zeros behind), and one call at a time uses it.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Optional

import torch

from . import (_I64, _VP, SSD_BF16, SSD_F32, SSDError, _check_cuda, _ptr, _stream_handle,
               load_library)

#: Steps between the states that the recurrence keeps for its backward pass.
GATED_RECURRENCE_CHUNK = 64

#: Bytes at the start of a workspace that are zero before its first call.
HEADER_BYTES = 256

ACTIVATIONS = {None: 0, "none": 0, "silu": 1}
_IO = {torch.float32: SSD_F32, torch.bfloat16: SSD_BF16}


class gated_recurrence_shape(ctypes.Structure):
    _fields_ = [("batch", _I64), ("seqlen", _I64), ("d_model", _I64), ("x_stride", _I64 * 2),
                ("gate_a_stride", _I64 * 2), ("gate_x_stride", _I64 * 2), ("dy_stride", _I64 * 2),
                ("c", ctypes.c_float), ("io_dtype", ctypes.c_int32)]


class group_norm_shape(ctypes.Structure):
    _fields_ = [("batch", _I64), ("rows", _I64), ("channels", _I64), ("groups", _I64),
                ("x_stride", _I64 * 2), ("dy_stride", _I64 * 2), ("eps", ctypes.c_float),
                ("activation", ctypes.c_int32), ("io_dtype", ctypes.c_int32)]


def _declare(lib) -> None:
    """Result and argument types of this module's C functions."""
    size, i32, f32 = ctypes.c_size_t, ctypes.c_int32, ctypes.c_float
    R, G = ctypes.POINTER(gated_recurrence_shape), ctypes.POINTER(group_norm_shape)
    for name, res, args in (
            ("gated_recurrence_workspace_bytes", size, [R, i32]),
            ("gated_recurrence_forward", ctypes.c_int, [R] + [_VP] * 9 + [size, _VP]),
            ("gated_recurrence_backward", ctypes.c_int, [R] + [_VP] * 14 + [size, _VP]),
            ("gated_recurrence_step", ctypes.c_int, [R] + [_VP] * 8),
            ("group_norm_workspace_bytes", size, [G, i32]),
            ("group_norm_forward", ctypes.c_int, [G] + [_VP] * 7 + [size, _VP]),
            ("group_norm_backward", ctypes.c_int, [G] + [_VP] * 10 + [size, _VP]),
            ("embedding_forward", ctypes.c_int,
             [_VP, i32, _I64, _VP, _I64, _I64, i32, f32, _VP, _VP]),
            ("embedding_backward_workspace_bytes", size, [_I64] * 3),
            ("embedding_backward", ctypes.c_int,
             [_VP, i32, _I64, _VP, _I64, _I64, i32, f32, _VP, _VP, size, _VP])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args


def _check_rows(name, t, dtype, shape):
    """As _check_cuda, for a tensor of any strides whose last axis is contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous along its last axis")


def _io_dtype(name, t):
    if isinstance(t, torch.Tensor) and t.dtype not in _IO:
        raise ValueError(f"{name} must be float32 or bfloat16")


def _strides(t, axes):
    """Strides of `axes`; an axis of one element (or none) has stride 0."""
    return (_I64 * 2)(*(t.stride(a) if t.shape[a] > 1 else 0 for a in axes))


class _Plan:
    """What the plans share: the buffers of one call, on one device and one stream."""

    _name = ""

    def _begin(self, device, stream):
        if device.index != torch.cuda.current_device():
            raise ValueError(f"tensors are on {device}, not on the current CUDA device")
        self._lib = load_library()
        self._device, self._stream, self._given = device, stream, []
        return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)

    def _out(self, name, given, dtype, shape):
        if given is None:
            return torch.empty(shape, dtype=dtype, device=self._device)
        _check_cuda(name, given, dtype, shape)
        self._passed(name, given)
        return given

    def _passed(self, name, given):
        """A buffer of the caller's that the call writes."""
        if given.device != self._device:
            raise ValueError(f"{name} must be on {self._device}, got {given.device}")
        self._given.append(given)

    def _workspace(self, given, need, what):
        if need == 0:
            raise SSDError(2, f"{what} (sizes not supported)")
        if given is None:
            given = torch.empty(need, dtype=torch.uint8, device=self._device)
            given[:HEADER_BYTES].zero_()
            return given
        _check_cuda("workspace", given, torch.uint8)
        self._passed("workspace", given)
        return given

    def _finish(self, inputs, args):
        """Keeps the inputs alive as long as the plan, on the plan's device and stream."""
        self.inputs = tuple(t for t in inputs if t is not None)
        for t in self.inputs:
            if t.device != self._device:
                raise ValueError(f"all tensors must be on {self._device}, one is on {t.device}")
        if self._stream is not None:
            for t in (*self.inputs, *self._given):
                t.record_stream(self._stream)
        self._args = (*args, _stream_handle(self._stream))
        self._fn = getattr(self._lib, self._name)

    def _call(self):
        st = self._fn(*self._args)
        if st != 0:
            raise SSDError(st, self._name)


def _recurrence_shape(x, gate_a, gate_x, dy, c) -> gated_recurrence_shape:
    b, T, D = x.shape
    return gated_recurrence_shape(b, T, D, *(_strides(t, (0, 1)) for t in (x, gate_a, gate_x)),
                                  (_I64 * 2)() if dy is None else _strides(dy, (0, 1)), float(c),
                                  _IO[x.dtype])


def _check_recurrence(x, gate_a, gate_x, decay, init_state, c, dims=3):
    if not isinstance(x, torch.Tensor) or x.dim() != dims:
        raise ValueError("x must be [b,T,D]" if dims == 3 else "x must be [b,D]")
    _io_dtype("x", x)
    _check_rows("x", x, None, x.shape)
    _check_rows("gate_a", gate_a, x.dtype, x.shape)
    _check_rows("gate_x", gate_x, x.dtype, x.shape)
    _check_cuda("decay", decay, torch.float32, (x.shape[-1],))
    if init_state is not None:
        _check_cuda("init_state", init_state, torch.float32, (x.shape[0], x.shape[-1]))
    if not (c > 0 and math.isfinite(c)):
        raise ValueError(f"c must be positive and finite, got {c}")


class GatedRecurrencePlan(_Plan):
    """Arguments of ``gated_recurrence_forward`` checked once, for repeated calls on the same
    buffers; calling the plan returns (y, final_state, states)."""

    _name = "gated_recurrence_forward"

    def __init__(self, x, gate_a, gate_x, decay, *, c: float = 8.0, init_state=None, y=None,
                 final_state=None, return_final_state: bool = True, states=None,
                 return_states: bool = False, workspace=None, stream=None):
        _check_recurrence(x, gate_a, gate_x, decay, init_state, c)
        b, T, D = x.shape
        self.shape = _recurrence_shape(x, gate_a, gate_x, None, c)
        with self._begin(x.device, stream):
            self.y = self._out("y", y, x.dtype, (b, T, D))
            if return_final_state or final_state is not None:
                final_state = self._out("final_state", final_state, torch.float32, (b, D))
            if return_states or states is not None:
                states = self._out("states", states, torch.float32,
                                   (b, -(-T // GATED_RECURRENCE_CHUNK), D))
            need = int(self._lib.gated_recurrence_workspace_bytes(ctypes.byref(self.shape), 0))
            self.workspace = self._workspace(workspace, need, "gated_recurrence_workspace_bytes")
        self.final_state, self.states = final_state, states
        self._finish((x, gate_a, gate_x, decay, init_state),
                     (ctypes.byref(self.shape), _ptr(x), _ptr(gate_a), _ptr(gate_x), _ptr(decay),
                      _ptr(init_state), _ptr(self.y), _ptr(final_state), _ptr(states),
                      _ptr(self.workspace), ctypes.c_size_t(self.workspace.numel())))

    def __call__(self):
        self._call()
        return self.y, self.final_state, self.states


def gated_recurrence_forward(x, gate_a, gate_x, decay, *, c: float = 8.0, init_state=None, y=None,
                             final_state=None, return_final_state: bool = True, states=None,
                             return_states: bool = False, workspace=None, stream=None):
    """Gated linear recurrence through ``gated_recurrence_forward``:

        a = exp(-c softplus(decay) sigmoid(gate_a)),  h_t = a h_{t-1} + sqrt(1 - a^2) sigmoid(gate_x) x

    x, gate_a, gate_x [b,T,D] (all f32 or all bf16; any strides with a contiguous last axis), decay
    [D] f32, init_state [b,D] f32.  Returns (y, final_state, states): y = h [b,T,D] in x's dtype,
    final_state [b,D] f32 and, with ``return_states``, the states [b, ceil(T/64), D] f32 that
    ``gated_recurrence_backward`` takes (None where not requested)."""
    return GatedRecurrencePlan(x, gate_a, gate_x, decay, c=c, init_state=init_state, y=y,
                               final_state=final_state, return_final_state=return_final_state,
                               states=states, return_states=return_states, workspace=workspace,
                               stream=stream)()


class GatedRecurrenceBackwardPlan(_Plan):
    """Arguments of ``gated_recurrence_backward`` checked once; calling the plan returns the dict
    dx, dgate_a, dgate_x (x's dtype), ddecay and dinit (f32; dinit None unless return_dinit)."""

    _name = "gated_recurrence_backward"

    def __init__(self, x, gate_a, gate_x, decay, dy, *, c: float = 8.0, init_state=None,
                 states=None, dfinal=None, return_dinit: bool = True,
                 grads: Optional[dict] = None, workspace=None, stream=None):
        _check_recurrence(x, gate_a, gate_x, decay, init_state, c)
        b, T, D = x.shape
        _check_rows("dy", dy, x.dtype, x.shape)
        if states is not None:
            _check_cuda("states", states, torch.float32, (b, -(-T // GATED_RECURRENCE_CHUNK), D))
        if dfinal is not None:
            _check_cuda("dfinal", dfinal, torch.float32, (b, D))
        self.shape = _recurrence_shape(x, gate_a, gate_x, dy, c)
        g = dict(grads or {})
        with self._begin(x.device, stream):
            for k in ("dx", "dgate_a", "dgate_x"):
                g[k] = self._out(k, g.get(k), x.dtype, (b, T, D))
            g["ddecay"] = self._out("ddecay", g.get("ddecay"), torch.float32, (D,))
            g["dinit"] = (self._out("dinit", g.get("dinit"), torch.float32, (b, D))
                          if return_dinit else None)
            need = int(self._lib.gated_recurrence_workspace_bytes(ctypes.byref(self.shape), 1))
            self.workspace = self._workspace(workspace, need, "gated_recurrence_workspace_bytes")
        self.grads = g
        self._finish((x, gate_a, gate_x, decay, dy, init_state, states, dfinal),
                     (ctypes.byref(self.shape), _ptr(x), _ptr(gate_a), _ptr(gate_x), _ptr(decay),
                      _ptr(init_state), _ptr(states), _ptr(dy), _ptr(dfinal), _ptr(g["dx"]),
                      _ptr(g["dgate_a"]), _ptr(g["dgate_x"]), _ptr(g["ddecay"]), _ptr(g["dinit"]),
                      _ptr(self.workspace), ctypes.c_size_t(self.workspace.numel())))

    def __call__(self):
        self._call()
        return self.grads


def gated_recurrence_backward(x, gate_a, gate_x, decay, dy, *, c: float = 8.0, init_state=None,
                              states=None, dfinal=None, return_dinit: bool = True, grads=None,
                              workspace=None, stream=None):
    """Gradients of <dy, y> + <dfinal, final_state> for ``gated_recurrence_forward`` on the same
    inputs.  ``states`` is what the forward kept (``return_states``); without it the call recomputes
    it with one more pass over the inputs.  Returns a dict dx, dgate_a, dgate_x, ddecay, dinit."""
    return GatedRecurrenceBackwardPlan(x, gate_a, gate_x, decay, dy, c=c, init_state=init_state,
                                       states=states, dfinal=dfinal, return_dinit=return_dinit,
                                       grads=grads, workspace=workspace, stream=stream)()


class GatedRecurrenceStepPlan(_Plan):
    """Arguments of ``gated_recurrence_step`` checked once; calling the plan returns (y, state_out).
    Without ``state_out`` the state is updated in place."""

    _name = "gated_recurrence_step"

    def __init__(self, x, gate_a, gate_x, decay, state, *, c: float = 8.0, y=None, state_out=None,
                 stream=None):
        _check_recurrence(x, gate_a, gate_x, decay, state, c, dims=2)
        if state is None:
            raise ValueError("state must be a [b,D] float32 tensor")
        b, D = x.shape
        self.shape = gated_recurrence_shape(
            b, 1, D, *((_I64 * 2)(_strides(t, (0, 0))[0], 0) for t in (x, gate_a, gate_x)),
            (_I64 * 2)(), float(c), _IO[x.dtype])
        with self._begin(x.device, stream):
            self.y = self._out("y", y, x.dtype, (b, D))
            self.state_out = self._out("state_out", state if state_out is None else state_out,
                                       torch.float32, (b, D))
        self._finish((x, gate_a, gate_x, decay, state),
                     (ctypes.byref(self.shape), _ptr(x), _ptr(gate_a), _ptr(gate_x), _ptr(decay),
                      _ptr(state), _ptr(self.y), _ptr(self.state_out)))

    def __call__(self):
        self._call()
        return self.y, self.state_out


def gated_recurrence_step(x, gate_a, gate_x, decay, state, *, c: float = 8.0, y=None,
                          state_out=None, stream=None):
    """One step of the recurrence for every sequence of a batch (serving): x, gate_a, gate_x [b,D],
    state [b,D] f32, updated in place unless ``state_out`` is given.  Returns (y, state)."""
    return GatedRecurrenceStepPlan(x, gate_a, gate_x, decay, state, c=c, y=y, state_out=state_out,
                                   stream=stream)()


def _norm_view(name, t):
    """t as [N,S,C] without a copy: [N,C], [N,S,C] with any outer strides, or contiguous [N,...,C]."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() < 2:
        raise ValueError(f"{name} must be [N,C] or [N,...,C]")
    if t.dim() == 2:
        return t.unsqueeze(1)
    if t.dim() == 3:
        return t
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (or [N,S,C] with a contiguous last axis)")
    return t.view(t.shape[0], math.prod(t.shape[1:-1]), t.shape[-1])


def _norm_shape(x, dy, groups, eps, activation) -> group_norm_shape:
    N, S, C = x.shape
    return group_norm_shape(N, S, C, int(groups), _strides(x, (0, 1)),
                            (_I64 * 2)() if dy is None else _strides(dy, (0, 1)), float(eps),
                            ACTIVATIONS[activation], _IO[x.dtype])


def _check_norm(x, num_groups, weight, bias, eps, activation):
    _io_dtype("x", x)
    _check_rows("x", x, None, x.shape)
    C = x.shape[-1]
    if num_groups < 1 or C < 1 or C % num_groups:
        raise ValueError(f"num_groups must divide the {C} channels, got {num_groups}")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(map(str, ACTIVATIONS))}")
    if not (eps >= 0 and math.isfinite(eps)):
        raise ValueError(f"eps must be finite and not negative, got {eps}")
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            _check_cuda(name, t, torch.float32, (C,))


class GroupNormPlan(_Plan):
    """Arguments of ``group_norm_forward`` checked once; calling the plan returns (y, mean, rstd)."""

    _name = "group_norm_forward"

    def __init__(self, x, num_groups: int, weight=None, bias=None, *, eps: float = 1e-5,
                 activation: Optional[str] = "silu", y=None, mean=None, rstd=None, workspace=None,
                 stream=None):
        v = _norm_view("x", x)
        _check_norm(v, num_groups, weight, bias, eps, activation)
        self.shape = _norm_shape(v, None, num_groups, eps, activation)
        with self._begin(x.device, stream):
            self.y = self._out("y", y, x.dtype, tuple(x.shape))
            self.mean = self._out("mean", mean, torch.float32, (v.shape[0], num_groups))
            self.rstd = self._out("rstd", rstd, torch.float32, (v.shape[0], num_groups))
            need = int(self._lib.group_norm_workspace_bytes(ctypes.byref(self.shape), 0))
            self.workspace = self._workspace(workspace, need, "group_norm_workspace_bytes")
        self._finish((x, weight, bias),
                     (ctypes.byref(self.shape), _ptr(x), _ptr(weight), _ptr(bias), _ptr(self.y),
                      _ptr(self.mean), _ptr(self.rstd), _ptr(self.workspace),
                      ctypes.c_size_t(self.workspace.numel())))

    def __call__(self):
        self._call()
        return self.y, self.mean, self.rstd


def group_norm_forward(x, num_groups: int, weight=None, bias=None, *, eps: float = 1e-5,
                       activation: Optional[str] = "silu", y=None, mean=None, rstd=None,
                       workspace=None, stream=None):
    """Group norm with an activation, channels last, through ``group_norm_forward``.

    x [N,C], [N,S,C] (any strides with a contiguous last axis) or contiguous [N,...,C], f32 or bf16;
    the statistics of a sample's group run over all its positions and its C/num_groups neighbouring
    channels.  weight, bias [C] f32 (None: ones, zeros); activation "silu" or None.  Returns (y,
    mean, rstd) with mean, rstd [N, num_groups] f32 for ``group_norm_backward``.  [N,C] is the norm
    of every token's heads after a scan."""
    return GroupNormPlan(x, num_groups, weight, bias, eps=eps, activation=activation, y=y,
                         mean=mean, rstd=rstd, workspace=workspace, stream=stream)()


class GroupNormBackwardPlan(_Plan):
    """Arguments of ``group_norm_backward`` checked once; calling the plan returns the dict dx (x's
    dtype), dweight and dbias (f32; None without ``param_grads``)."""

    _name = "group_norm_backward"

    def __init__(self, x, dy, num_groups: int, mean, rstd, weight=None, bias=None, *,
                 activation: Optional[str] = "silu", param_grads: bool = True,
                 grads: Optional[dict] = None, workspace=None, stream=None):
        v, dv = _norm_view("x", x), _norm_view("dy", dy)
        _check_norm(v, num_groups, weight, bias, 0.0, activation)
        _check_rows("dy", dy, x.dtype, x.shape)
        for name, t in (("mean", mean), ("rstd", rstd)):
            _check_cuda(name, t, torch.float32, (v.shape[0], num_groups))
        self.shape = _norm_shape(v, dv, num_groups, 0.0, activation)
        g = dict(grads or {})
        with self._begin(x.device, stream):
            g["dx"] = self._out("dx", g.get("dx"), x.dtype, tuple(x.shape))
            for k in ("dweight", "dbias"):
                g[k] = (self._out(k, g.get(k), torch.float32, (x.shape[-1],))
                        if param_grads else None)
            need = int(self._lib.group_norm_workspace_bytes(ctypes.byref(self.shape), 1))
            self.workspace = self._workspace(workspace, need, "group_norm_workspace_bytes")
        self.grads = g
        self._finish((x, dy, mean, rstd, weight, bias),
                     (ctypes.byref(self.shape), _ptr(x), _ptr(dy), _ptr(mean), _ptr(rstd),
                      _ptr(weight), _ptr(bias), _ptr(g["dx"]), _ptr(g["dweight"]),
                      _ptr(g["dbias"]), _ptr(self.workspace),
                      ctypes.c_size_t(self.workspace.numel())))

    def __call__(self):
        self._call()
        return self.grads


def group_norm_backward(x, dy, num_groups: int, mean, rstd, weight=None, bias=None, *,
                        activation: Optional[str] = "silu", param_grads: bool = True, grads=None,
                        workspace=None, stream=None):
    """Gradients of <dy, y> for ``group_norm_forward`` on the same inputs; mean and rstd are what it
    returned.  Returns a dict dx, dweight, dbias."""
    return GroupNormBackwardPlan(x, dy, num_groups, mean, rstd, weight, bias,
                                 activation=activation, param_grads=param_grads, grads=grads,
                                 workspace=workspace, stream=stream)()


def _check_ids(ids):
    _check_cuda("ids", ids)
    if ids.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"ids must be int32 or int64, got {ids.dtype}")
    return 32 if ids.dtype == torch.int32 else 64


class EmbeddingPlan(_Plan):
    """Arguments of ``embedding_forward`` checked once; calling the plan returns out."""

    _name = "embedding_forward"

    def __init__(self, ids, table, *, scale: float = 1.0, out=None, stream=None):
        bits = _check_ids(ids)
        _check_cuda("table", table)
        _io_dtype("table", table)
        if table.dim() != 2 or 0 in table.shape:
            raise ValueError("table must be [V,D] with at least one row and one column")
        V, D = table.shape
        with self._begin(table.device, stream):
            self.out = self._out("out", out, table.dtype, (*ids.shape, D))
        self._finish((ids, table),
                     (_ptr(ids), bits, ids.numel(), _ptr(table), V, D, _IO[table.dtype],
                      ctypes.c_float(scale), _ptr(self.out)))

    def __call__(self):
        self._call()
        return self.out


def embedding_forward(ids, table, *, scale: float = 1.0, out=None, stream=None):
    """Rows of ``table`` [V,D] (f32 or bf16) times ``scale`` for ids of any shape (int32 or int64)
    through ``embedding_forward``; an id outside [0,V) is padding and gives zeros."""
    return EmbeddingPlan(ids, table, scale=scale, out=out, stream=stream)()


class EmbeddingBackwardPlan(_Plan):
    """Arguments of ``embedding_backward`` checked once; calling the plan returns dtable [V,D] f32."""

    _name = "embedding_backward"

    def __init__(self, ids, dout, num_rows: int, *, scale: float = 1.0, dtable=None,
                 workspace=None, stream=None):
        bits = _check_ids(ids)
        _check_cuda("dout", dout)
        _io_dtype("dout", dout)
        if dout.dim() != ids.dim() + 1 or dout.shape[:-1] != ids.shape or dout.shape[-1] < 1:
            raise ValueError("dout must have the ids' shape and one more axis")
        V, D = int(num_rows), dout.shape[-1]
        if V < 1:
            raise ValueError(f"num_rows must be at least 1, got {num_rows}")
        n = ids.numel()
        with self._begin(dout.device, stream):
            self.dtable = self._out("dtable", dtable, torch.float32, (V, D))
            need = int(self._lib.embedding_backward_workspace_bytes(n, V, D))
            self.workspace = self._workspace(workspace, need, "embedding_backward_workspace_bytes")
        self._finish((ids, dout),
                     (_ptr(ids), bits, n, _ptr(dout), V, D, _IO[dout.dtype],
                      ctypes.c_float(scale), _ptr(self.dtable), _ptr(self.workspace),
                      ctypes.c_size_t(self.workspace.numel())))

    def __call__(self):
        self._call()
        return self.dtable


def embedding_backward(ids, dout, num_rows: int, *, scale: float = 1.0, dtable=None,
                       workspace=None, stream=None):
    """Gradient of ``embedding_forward`` with respect to its table: [num_rows, D] f32, every row
    written, each the sum of its tokens' dout rows times ``scale`` in an order that depends only on
    the ids (the same bits every run)."""
    return EmbeddingBackwardPlan(ids, dout, num_rows, scale=scale, dtable=dtable,
                                 workspace=workspace, stream=stream)()
