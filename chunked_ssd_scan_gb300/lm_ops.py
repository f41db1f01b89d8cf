"""Operators around a scan in a recurrent language model: the gated linear recurrence, the
channels-last group norm with an activation, the token embedding, the gated delta rule, the
root-mean-square norm with the residual's addition and an 8-bit output, and the drawing of tokens
(declarations and contracts in include/ssdscan.h).

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

#: Steps between the states that the delta rule keeps for its backward pass.
GATED_DELTA_RULE_CHUNK = 64

#: Channels that share a scale where the norm's 8-bit output has scales for blocks.
RMS_NORM_BLOCK = 128

ACTIVATIONS = {None: 0, "none": 0, "silu": 1}
QUANTIZE = {None: 0, "none": 0, "token": 1, "block": 2}
_IO = {torch.float32: SSD_F32, torch.bfloat16: SSD_BF16}


class gated_recurrence_shape(ctypes.Structure):
    _fields_ = [("batch", _I64), ("seqlen", _I64), ("d_model", _I64), ("x_stride", _I64 * 2),
                ("gate_a_stride", _I64 * 2), ("gate_x_stride", _I64 * 2), ("dy_stride", _I64 * 2),
                ("c", ctypes.c_float), ("io_dtype", ctypes.c_int32)]


class group_norm_shape(ctypes.Structure):
    _fields_ = [("batch", _I64), ("rows", _I64), ("channels", _I64), ("groups", _I64),
                ("x_stride", _I64 * 2), ("dy_stride", _I64 * 2), ("eps", ctypes.c_float),
                ("activation", ctypes.c_int32), ("io_dtype", ctypes.c_int32)]


class gated_delta_rule_shape(ctypes.Structure):
    _fields_ = [("batch", _I64), ("seqlen", _I64), ("key_heads", _I64), ("heads", _I64),
                ("key_dim", _I64), ("value_dim", _I64), ("q_stride", _I64 * 3),
                ("k_stride", _I64 * 3), ("v_stride", _I64 * 3), ("dy_stride", _I64 * 3),
                ("g_stride", _I64 * 2), ("beta_stride", _I64 * 2), ("scale", ctypes.c_float),
                ("io_dtype", ctypes.c_int32)]


class rms_norm_shape(ctypes.Structure):
    _fields_ = [("rows", _I64), ("channels", _I64), ("x_stride", _I64), ("res_stride", _I64),
                ("dy_stride", _I64), ("eps", ctypes.c_float), ("quantize", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32)]


class token_sample_shape(ctypes.Structure):
    _fields_ = [("rows", _I64), ("vocab", _I64), ("logits_stride", _I64),
                ("temperature", ctypes.c_float), ("top_p", ctypes.c_float),
                ("min_p", ctypes.c_float), ("top_k", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32)]


def _declare(lib) -> None:
    """Result and argument types of this module's C functions."""
    size, i32, f32 = ctypes.c_size_t, ctypes.c_int32, ctypes.c_float
    R, G = ctypes.POINTER(gated_recurrence_shape), ctypes.POINTER(group_norm_shape)
    D, N = ctypes.POINTER(gated_delta_rule_shape), ctypes.POINTER(rms_norm_shape)
    S = ctypes.POINTER(token_sample_shape)
    for name, res, args in (
            ("gated_delta_rule_workspace_bytes", size, [D, i32]),
            ("gated_delta_rule_forward", ctypes.c_int, [D] + [_VP] * 10 + [size, _VP]),
            ("gated_delta_rule_backward", ctypes.c_int, [D] + [_VP] * 16 + [size, _VP]),
            ("gated_delta_rule_step", ctypes.c_int, [D] + [_VP] * 9),
            ("rms_norm_workspace_bytes", size, [N]),
            ("rms_norm_forward", ctypes.c_int, [N] + [_VP] * 8),
            ("rms_norm_backward", ctypes.c_int, [N] + [_VP] * 8 + [size, _VP]),
            ("token_sample", ctypes.c_int, [S] + [_VP] * 9),
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


def _strides3(t, axes):
    """Strides of three axes; an axis of one element (or none) has stride 0."""
    return (_I64 * 3)(*(0 if a is None or t.shape[a] <= 1 else t.stride(a) for a in axes))


def _check_delta(q, k, v, g, beta, init_state, scale, step=False):
    lead = "[b" if step else "[b,T"
    if not isinstance(q, torch.Tensor) or q.dim() != (3 if step else 4):
        raise ValueError(f"q must be {lead},Hk,K]")
    if not isinstance(v, torch.Tensor) or v.dim() != q.dim():
        raise ValueError(f"v must be {lead},H,V]")
    _io_dtype("q", q)
    Hk, K, H, V = *q.shape[-2:], *v.shape[-2:]
    if min(Hk, K, H, V) < 1 or H % Hk:
        raise ValueError(f"the {Hk} key heads must divide the {H} heads, and no head be empty")
    if K > 256:
        raise ValueError(f"a key head has at most 256 channels, got {K}")
    _check_rows("q", q, None, q.shape)
    _check_rows("k", k, q.dtype, q.shape)
    _check_rows("v", v, q.dtype, (*q.shape[:-2], H, V))
    for name, t in (("g", g), ("beta", beta)):
        if t is not None or name == "beta":
            _check_rows(name, t, torch.float32, (*q.shape[:-2], H))
    if init_state is not None:
        _check_cuda("init_state", init_state, torch.float32, (q.shape[0], H, V, K))
    scale = K ** -0.5 if scale is None else float(scale)
    if not math.isfinite(scale):
        raise ValueError(f"scale must be finite, got {scale}")
    return scale


def _delta_shape(q, k, v, g, beta, dy, scale, step=False) -> gated_delta_rule_shape:
    axes = (0, None, 1) if step else (0, 1, 2)
    three = lambda t: _strides3(t, axes)   # noqa: E731
    two = lambda t: (_I64 * 2)(*_strides3(t, (*axes[:2], None))[:2])   # noqa: E731
    return gated_delta_rule_shape(
        q.shape[0], 1 if step else q.shape[1], q.shape[-2], v.shape[-2], q.shape[-1], v.shape[-1],
        three(q), three(k), three(v), (_I64 * 3)() if dy is None else three(dy),
        (_I64 * 2)() if g is None else two(g), two(beta), scale, _IO[q.dtype])


class GatedDeltaRulePlan(_Plan):
    """Arguments of ``gated_delta_rule_forward`` checked once, for repeated calls on the same
    buffers; calling the plan returns (y, final_state, states)."""

    _name = "gated_delta_rule_forward"

    def __init__(self, q, k, v, g, beta, *, scale: Optional[float] = None, init_state=None, y=None,
                 final_state=None, return_final_state: bool = True, states=None,
                 return_states: bool = False, workspace=None, stream=None):
        scale = _check_delta(q, k, v, g, beta, init_state, scale)
        b, T, H, V = v.shape
        K = q.shape[-1]
        self.shape = _delta_shape(q, k, v, g, beta, None, scale)
        with self._begin(q.device, stream):
            self.y = self._out("y", y, q.dtype, (b, T, H, V))
            if return_final_state or final_state is not None:
                final_state = self._out("final_state", final_state, torch.float32, (b, H, V, K))
            if return_states or states is not None:
                states = self._out("states", states, torch.float32,
                                   (b, -(-T // GATED_DELTA_RULE_CHUNK), H, V, K))
            need = int(self._lib.gated_delta_rule_workspace_bytes(ctypes.byref(self.shape), 0))
            self.workspace = self._workspace(workspace, need, "gated_delta_rule_workspace_bytes")
        self.final_state, self.states = final_state, states
        self._finish((q, k, v, g, beta, init_state),
                     (ctypes.byref(self.shape), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                      _ptr(init_state), _ptr(self.y), _ptr(final_state), _ptr(states),
                      _ptr(self.workspace), ctypes.c_size_t(self.workspace.numel())))

    def __call__(self):
        self._call()
        return self.y, self.final_state, self.states


def gated_delta_rule_forward(q, k, v, g, beta, *, scale: Optional[float] = None, init_state=None,
                             y=None, final_state=None, return_final_state: bool = True,
                             states=None, return_states: bool = False, workspace=None,
                             stream=None):
    """Gated delta rule through ``gated_delta_rule_forward``, for every sequence and head a state
    S [V,K]:

        S = exp(g_t) S;  S = S + beta_t (v_t - S k_t) k_t^T;  y_t = scale S q_t

    q, k [b,T,Hk,K] and v [b,T,H,V] (all f32 or all bf16; any strides with a contiguous last axis;
    head h reads q and k of h // (H / Hk)), g (None: zeros) and beta [b,T,H] f32, init_state
    [b,H,V,K] f32; scale is K^-1/2 unless given.  Returns (y, final_state, states): y [b,T,H,V] in
    q's dtype, final_state f32 and, with ``return_states``, the states [b, ceil(T/64), H, V, K] f32
    that ``gated_delta_rule_backward`` takes (None where not requested).  final_state and states
    must not lie over init_state (SSDError)."""
    return GatedDeltaRulePlan(q, k, v, g, beta, scale=scale, init_state=init_state, y=y,
                              final_state=final_state, return_final_state=return_final_state,
                              states=states, return_states=return_states, workspace=workspace,
                              stream=stream)()


class GatedDeltaRuleBackwardPlan(_Plan):
    """Arguments of ``gated_delta_rule_backward`` checked once; calling the plan returns the dict
    dq, dk, dv (q's dtype), dg (None where g is), dbeta and dinit (f32; None unless
    return_dinit)."""

    _name = "gated_delta_rule_backward"

    def __init__(self, q, k, v, g, beta, dy, *, scale: Optional[float] = None, init_state=None,
                 states=None, dfinal=None, return_dinit: bool = True,
                 grads: Optional[dict] = None, workspace=None, stream=None):
        scale = _check_delta(q, k, v, g, beta, init_state, scale)
        b, T, H, V = v.shape
        K = q.shape[-1]
        _check_rows("dy", dy, q.dtype, v.shape)
        if states is not None:
            _check_cuda("states", states, torch.float32,
                        (b, -(-T // GATED_DELTA_RULE_CHUNK), H, V, K))
        if dfinal is not None:
            _check_cuda("dfinal", dfinal, torch.float32, (b, H, V, K))
        self.shape = _delta_shape(q, k, v, g, beta, dy, scale)
        out = dict(grads or {})
        with self._begin(q.device, stream):
            for name, like in (("dq", q), ("dk", q), ("dv", v)):
                out[name] = self._out(name, out.get(name), q.dtype, tuple(like.shape))
            out["dg"] = (None if g is None else
                         self._out("dg", out.get("dg"), torch.float32, (b, T, H)))
            out["dbeta"] = self._out("dbeta", out.get("dbeta"), torch.float32, (b, T, H))
            out["dinit"] = (self._out("dinit", out.get("dinit"), torch.float32, (b, H, V, K))
                            if return_dinit else None)
            need = int(self._lib.gated_delta_rule_workspace_bytes(ctypes.byref(self.shape), 1))
            self.workspace = self._workspace(workspace, need, "gated_delta_rule_workspace_bytes")
        self.grads = out
        self._finish((q, k, v, g, beta, dy, init_state, states, dfinal),
                     (ctypes.byref(self.shape), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                      _ptr(init_state), _ptr(states), _ptr(dy), _ptr(dfinal), _ptr(out["dq"]),
                      _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dg"]), _ptr(out["dbeta"]),
                      _ptr(out["dinit"]), _ptr(self.workspace),
                      ctypes.c_size_t(self.workspace.numel())))

    def __call__(self):
        self._call()
        return self.grads


def gated_delta_rule_backward(q, k, v, g, beta, dy, *, scale: Optional[float] = None,
                              init_state=None, states=None, dfinal=None,
                              return_dinit: bool = True, grads=None, workspace=None, stream=None):
    """Gradients of <dy, y> + <dfinal, final_state> for ``gated_delta_rule_forward`` on the same
    inputs.  ``states`` is what the forward kept (``return_states``); without it the call recomputes
    it.  Returns a dict dq, dk (summed over the heads that share them), dv, dg, dbeta, dinit."""
    return GatedDeltaRuleBackwardPlan(q, k, v, g, beta, dy, scale=scale, init_state=init_state,
                                      states=states, dfinal=dfinal, return_dinit=return_dinit,
                                      grads=grads, workspace=workspace, stream=stream)()


class GatedDeltaRuleStepPlan(_Plan):
    """Arguments of ``gated_delta_rule_step`` checked once; calling the plan returns (y, state_out).
    Without ``state_out`` the state is updated in place."""

    _name = "gated_delta_rule_step"

    def __init__(self, q, k, v, g, beta, state, *, scale: Optional[float] = None, y=None,
                 state_out=None, stream=None):
        if state is None:
            raise ValueError("state must be a [b,H,V,K] float32 tensor")
        scale = _check_delta(q, k, v, g, beta, state, scale, step=True)
        self.shape = _delta_shape(q, k, v, g, beta, None, scale, step=True)
        with self._begin(q.device, stream):
            self.y = self._out("y", y, q.dtype, tuple(v.shape))
            self.state_out = self._out("state_out", state if state_out is None else state_out,
                                       torch.float32, tuple(state.shape))
        self._finish((q, k, v, g, beta, state),
                     (ctypes.byref(self.shape), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                      _ptr(state), _ptr(self.y), _ptr(self.state_out)))

    def __call__(self):
        self._call()
        return self.y, self.state_out


def gated_delta_rule_step(q, k, v, g, beta, state, *, scale: Optional[float] = None, y=None,
                          state_out=None, stream=None):
    """One step of the rule for every sequence of a batch (serving): q, k [b,Hk,K], v [b,H,V], g
    (None: zeros), beta [b,H], state [b,H,V,K] f32, updated in place unless ``state_out`` is given.
    Returns (y, state)."""
    return GatedDeltaRuleStepPlan(q, k, v, g, beta, state, scale=scale, y=y, state_out=state_out,
                                  stream=stream)()


def _row_view(name, t, like=None):
    """t as [N,C] without a copy: [N,C] with any row stride, or contiguous [...,C]."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if like is not None and tuple(t.shape) != tuple(like.shape):
        raise ValueError(f"{name} must have shape {tuple(like.shape)}, got {tuple(t.shape)}")
    if t.dim() < 1 or t.shape[-1] < 1:
        raise ValueError(f"{name} must be [...,C] with at least one channel")
    if t.dim() == 2:
        return t
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (or [N,C] with a contiguous last axis)")
    return t.view(math.prod(t.shape[:-1]), t.shape[-1])


def _rms_shape(x, res, dy, eps, quantize) -> rms_norm_shape:
    stride = lambda t: 0 if t is None or t.shape[0] <= 1 else t.stride(0)   # noqa: E731
    return rms_norm_shape(*x.shape, stride(x), stride(res), stride(dy), float(eps),
                          QUANTIZE[quantize], _IO[x.dtype])


class RMSNormPlan(_Plan):
    """Arguments of ``rms_norm_forward`` checked once; calling the plan returns (y, h, rstd,
    scale)."""

    _name = "rms_norm_forward"

    def __init__(self, x, weight=None, *, residual=None, eps: float = 1e-6,
                 quantize: Optional[str] = None, y=None, h=None, rstd=None, scale=None,
                 stream=None):
        v = _row_view("x", x)
        _io_dtype("x", x)
        _check_rows("x", v, None, v.shape)
        r = None
        if residual is not None:
            r = _row_view("residual", residual, x)
            _check_rows("residual", r, x.dtype, v.shape)
        if quantize not in QUANTIZE:
            raise ValueError(f"quantize must be one of {sorted(map(str, QUANTIZE))}")
        if not (eps >= 0 and math.isfinite(eps)):
            raise ValueError(f"eps must be finite and not negative, got {eps}")
        N, C = v.shape
        if weight is not None:
            _check_cuda("weight", weight, torch.float32, (C,))
        kind = QUANTIZE[quantize]
        if scale is not None and not kind:
            raise ValueError("scale is an output of an 8-bit y only")
        self.shape = _rms_shape(v, r, None, eps, quantize)
        with self._begin(x.device, stream):
            self.y = self._out("y", y, torch.float8_e4m3fn if kind else x.dtype, tuple(x.shape))
            if residual is not None or h is not None:
                h = self._out("h", h, x.dtype, tuple(x.shape))
            self.rstd = self._out("rstd", rstd, torch.float32, tuple(x.shape[:-1]))
            if kind:
                scale = self._out("scale", scale, torch.float32,
                                  (*x.shape[:-1], 1 if kind == 1 else -(-C // RMS_NORM_BLOCK)))
        self.h, self.scale = h, scale
        self._finish((x, residual, weight),
                     (ctypes.byref(self.shape), _ptr(x), _ptr(residual), _ptr(weight),
                      _ptr(self.y), _ptr(h), _ptr(self.rstd), _ptr(scale)))

    def __call__(self):
        self._call()
        return self.y, self.h, self.rstd, self.scale


def rms_norm_forward(x, weight=None, *, residual=None, eps: float = 1e-6,
                     quantize: Optional[str] = None, y=None, h=None, rstd=None, scale=None,
                     stream=None):
    """Root-mean-square norm of every row, after the residual's addition, through
    ``rms_norm_forward``:

        h = x + residual;  y = h / sqrt(mean(h^2) + eps) * weight

    x and residual [N,C] (any row stride) or contiguous [...,C], f32 or bf16; weight [C] f32 (None:
    ones).  Returns (y, h, rstd, scale): h (None without a residual) is the sum in x's dtype, the
    residual of the next layer; rstd [...] f32 is for ``rms_norm_backward``.  With ``quantize``
    "token" or "block" y is float8_e4m3fn and stands for y * scale, with a scale f32 [...,1] for
    every row or [..., ceil(C/128)] for every 128 channels (None otherwise)."""
    return RMSNormPlan(x, weight, residual=residual, eps=eps, quantize=quantize, y=y, h=h,
                       rstd=rstd, scale=scale, stream=stream)()


class RMSNormBackwardPlan(_Plan):
    """Arguments of ``rms_norm_backward`` checked once; calling the plan returns the dict dx (h's
    dtype) and dweight (f32; None without ``param_grads``)."""

    _name = "rms_norm_backward"

    def __init__(self, h, dy, rstd, weight=None, *, dresidual=None, param_grads: bool = True,
                 grads: Optional[dict] = None, workspace=None, stream=None):
        v = _row_view("h", h)
        _io_dtype("h", h)
        _check_rows("h", v, None, v.shape)
        d = _row_view("dy", dy, h)
        _check_rows("dy", d, h.dtype, v.shape)
        r = None
        if dresidual is not None:
            r = _row_view("dresidual", dresidual, h)
            _check_rows("dresidual", r, h.dtype, v.shape)
        N, C = v.shape
        _check_cuda("rstd", rstd, torch.float32, tuple(h.shape[:-1]))
        if weight is not None:
            _check_cuda("weight", weight, torch.float32, (C,))
        self.shape = _rms_shape(v, r, d, 0.0, None)
        g = dict(grads or {})
        with self._begin(h.device, stream):
            g["dx"] = self._out("dx", g.get("dx"), h.dtype, tuple(h.shape))
            g["dweight"] = (self._out("dweight", g.get("dweight"), torch.float32, (C,))
                            if param_grads else None)
            need = int(self._lib.rms_norm_workspace_bytes(ctypes.byref(self.shape)))
            self.workspace = self._workspace(workspace, need, "rms_norm_workspace_bytes")
        self.grads = g
        self._finish((h, dy, rstd, weight, dresidual),
                     (ctypes.byref(self.shape), _ptr(h), _ptr(dy), _ptr(rstd), _ptr(weight),
                      _ptr(dresidual), _ptr(g["dx"]), _ptr(g["dweight"]), _ptr(self.workspace),
                      ctypes.c_size_t(self.workspace.numel())))

    def __call__(self):
        self._call()
        return self.grads


def rms_norm_backward(h, dy, rstd, weight=None, *, dresidual=None, param_grads: bool = True,
                      grads=None, workspace=None, stream=None):
    """Gradients of <dy, y> + <dresidual, h> for ``rms_norm_forward``; h and rstd are what it
    returned (h is x where there was no residual).  Returns a dict dx, the gradient of x and of the
    residual alike, and dweight."""
    return RMSNormBackwardPlan(h, dy, rstd, weight, dresidual=dresidual, param_grads=param_grads,
                               grads=grads, workspace=workspace, stream=stream)()


class TokenSamplePlan(_Plan):
    """Arguments of ``token_sample`` checked once; calling the plan returns (ids, logprob)."""

    _name = "token_sample"

    def __init__(self, logits, u, *, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, ids=None,
                 logprob=None, stream=None):
        if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
            raise ValueError("logits must be [n,V]")
        _io_dtype("logits", logits)
        _check_rows("logits", logits, None, logits.shape)
        n, V = logits.shape
        if not 1 <= V <= 1 << 20:
            raise ValueError(f"logits must have 1 to {1 << 20} columns, got {V}")
        _check_cuda("u", u, torch.float32, (n,))
        given, plain = {}, {}
        for name, t, none, dtype in (("temperature", temperature, 1.0, torch.float32),
                                     ("top_k", top_k, 0, torch.int32),
                                     ("top_p", top_p, 1.0, torch.float32),
                                     ("min_p", min_p, 0.0, torch.float32)):
            given[name] = t if isinstance(t, torch.Tensor) else None
            plain[name] = none if t is None or given[name] is not None else t
            if given[name] is not None:
                _check_cuda(name, t, dtype, (n,))
        if not plain["temperature"] >= 0:
            raise ValueError(f"temperature must not be negative, got {temperature}")
        if plain["top_p"] != plain["top_p"] or plain["min_p"] != plain["min_p"]:
            raise ValueError("top_p and min_p must be numbers")
        self.shape = token_sample_shape(
            n, V, logits.stride(0) if n > 1 else 0, float(plain["temperature"]),
            float(plain["top_p"]), float(plain["min_p"]), min(max(int(plain["top_k"]), 0), V),
            _IO[logits.dtype])
        with self._begin(logits.device, stream):
            self.ids = self._out("ids", ids, torch.int64, (n,))
            self.logprob = self._out("logprob", logprob, torch.float32, (n,))
        self._finish((logits, u, *given.values()),
                     (ctypes.byref(self.shape), _ptr(logits), _ptr(u),
                      *(_ptr(given[k]) for k in ("temperature", "top_k", "top_p", "min_p")),
                      _ptr(self.ids), _ptr(self.logprob)))

    def __call__(self):
        self._call()
        return self.ids, self.logprob


def token_sample(logits, u, *, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, ids=None,
                 logprob=None, stream=None):
    """Draws one token for every row of logits [n,V] (f32 or bf16) from random numbers u [n] f32 in
    [0,1) through ``token_sample``.  Of the tokens by falling logit (equal ones by rising index) a
    row keeps the first ``top_k`` (<= 0: all), of these those of at least ``min_p`` times the
    largest probability, of these the fewest that hold ``top_p`` of their sum; the token drawn is
    the first by index at which the running sum of the kept weights exp(logit / temperature)
    exceeds u times their sum.  Temperature 0 takes the largest logit.  Each setting is a number or
    a tensor [n] (top_k int32, the others f32).  Returns (ids [n] int64, logprob [n] f32)."""
    return TokenSamplePlan(logits, u, temperature=temperature, top_k=top_k, top_p=top_p,
                           min_p=min_p, ids=ids, logprob=logprob, stream=stream)()
