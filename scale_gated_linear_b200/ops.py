"""Operators next to the MS-GLA layer, with their gradients and a form for single tokens.

gated_scan        the gated recurrence over sequences, one state per channel:
                      log a_t = logsigmoid(gate_t) / gate_normalizer
                      h_t = a_t h_{t-1} + u_t,  u_t = x_t  or (tied)  (1 - a_t) x_t
gated_scan_step   the same for one token of every sequence, updating the state in place
group_norm        group normalisation, channels last, with an activation or an output gate

gated_scan and group_norm take part in autograd (backwards; forward-mode derivatives are
refused). The pairs gated_scan_forward /
gated_scan_backward and group_norm_forward / group_norm_backward do the same by hand:
the forward returns what its backward needs. Both forms run the kernels of libmsgla.so;
this module checks arguments, allocates outputs and workspaces, and passes pointers.

Tensors are cuda tensors of one device (not necessarily the current one). x, the gate and
their gradients share one dtype (bfloat16, float16 or float32); states, weights and
their gradients are float32. The last dimension is contiguous, the others may have any
strides (views of a fused projection, expanded tensors). The work is enqueued on `stream`
(default: torch's current stream of that device) and is not waited for. A call that breaks one of
these rules raises MSGLAError before anything is launched.

Capturing a backward pass into a CUDA graph: autograd adds a leaf's gradient on the stream
that was current when the leaf first joined a graph that still lives. If that is an eager
graph of the same leaf, the capture would break inside the autograd engine, so gated_scan
and group_norm refuse a captured call then. torch does not tell the stream of a node, so a
captured call is refused for every leaf whose node lives and was not first used by these
functions in that capture: a leaf that another operation of the same capture has used before
them, and a leaf whose node something holds for its whole life, as data-parallel wrappers do.
Drop the eager outputs first, or capture the explicit pairs, which keep autograd out.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional

import torch
from torch.autograd import forward_ad

from . import _lib
from ._lib import MSGLAError

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_ACTIVATIONS = {None: 0, "none": 0, "silu": 1, "sigmoid": 2}


def _refuse(message: str, status: int = -1):
    raise MSGLAError(status, message)


@functools.lru_cache(maxsize=256)
def _scan_config(device: int, dtype, D: int, tied: bool, gate_normalizer: float):
    return _lib.ScanConfig(device, _DTYPES[dtype], D, 1 if tied else 0, gate_normalizer)


@functools.lru_cache(maxsize=256)
def _norm_config(device: int, dtype, C: int, groups: int, activation, center: bool, eps: float):
    return _lib.NormConfig(device, _DTYPES[dtype], C, groups, _ACTIVATIONS[activation], 1 if center else 0, eps)


@functools.lru_cache(maxsize=8)
def _saved_rows(dtype) -> int:
    """Rows between two states that a forward saves, as the library keeps them."""
    n, L = ctypes.c_size_t(), 1 << 16
    _lib.check(_lib.load().msgla_scan_saved_size(_lib.ScanConfig(0, _DTYPES[dtype], 1, 0, 1.0), 1, L, ctypes.byref(n)))
    return 4 * L // n.value


def _number(name: str, v) -> float:
    """v as a Python number: the configurations are kept by value, and a tensor's can change."""
    try:
        return float(v)
    except (TypeError, ValueError, OverflowError, RuntimeError) as e:
        _refuse(f"{name}={v!r} must be a number ({e})")


def _check_x(name: str, t, dims: int):
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in _DTYPES and t.dim() == dims:
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _refuse(f"{name} must be a cuda tensor")
    if t.dtype not in _DTYPES:
        _refuse(f"{name} has dtype {t.dtype}: bfloat16, float16 or float32", -2)
    _refuse(f"{name} has {t.dim()} dimensions, {dims} are needed")


def _dual_level() -> bool:
    """Whether a level of forward-mode differentiation is open."""
    return getattr(forward_ad, "_current_level", 0) >= 0


def _refuse_tangents(name: str, *tensors):
    """In a dual level: a dual tensor's tangent would be dropped, which reads as a derivative of zero."""
    for t in tensors:
        if isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None:
            _refuse(f"{name} has no forward-mode derivatives", -2)


def _check_like(name: str, t, x):
    if not isinstance(t, torch.Tensor) or t.dtype is not x.dtype or t.shape != x.shape or t.device != x.device:
        _refuse(f"{name} must have the shape {tuple(x.shape)}, the dtype {x.dtype} and the device {x.device}")


def _check_f32(name: str, t, shape, device):
    if (not isinstance(t, torch.Tensor) or t.dtype is not torch.float32 or t.shape != shape or t.device != device
            or not t.is_contiguous()):
        _refuse(f"{name} must be a contiguous float32 tensor of shape {tuple(shape)} on {device}")


def _check_mask(mask, shape, device):
    if not isinstance(mask, torch.Tensor) or mask.shape != shape or mask.device != device:
        _refuse(f"mask must have the shape {tuple(shape)} and be on {device}")
    if mask.dtype not in (torch.bool, torch.uint8) or not mask.is_contiguous():
        _refuse("mask must be a contiguous bool or uint8 tensor")


def _rows3(name: str, t):
    """msgla_rows of t [B, L, C]."""
    sb, sl, sc = t.stride()
    if sc != 1 and t.shape[-1] > 1:
        _refuse(f"the last dimension of {name} must be contiguous")
    return _lib.Rows(t.data_ptr(), sb, sl)


def _rows2(name: str, t):
    """msgla_rows of t [N, C]: one row a sample."""
    sb, sc = t.stride()
    if sc != 1 and t.shape[1] > 1:
        _refuse(f"the last dimension of {name} must be contiguous")
    return _lib.Rows(t.data_ptr(), sb, 0)


def _ptr(t):
    return None if t is None else t.data_ptr()


# The handle of torch's current stream; a Stream object would take 2 us to make.
_current_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


class _On:
    """The stream of a call that named one: outputs are allocated for it, and inputs that the
    caller may free are kept from other streams until it has used them."""

    def __init__(self, device, stream, inputs):
        if stream.device != device:
            _refuse(f"the stream is on {stream.device}, the tensors are on {device}")
        self.stream, self.handle = stream, stream.cuda_stream
        if self.handle != _current_handle(device.index):
            for t in inputs:
                if t is not None:
                    t.record_stream(stream)

    def empty_like(self, t):
        with torch.cuda.stream(self.stream):
            return torch.empty_like(t, memory_format=torch.contiguous_format)

    def empty(self, shape, dtype, device):
        with torch.cuda.stream(self.stream):
            return torch.empty(shape, dtype=dtype, device=device)


class _Current:
    """A call on torch's current stream of its device."""
    __slots__ = ("handle",)

    def __init__(self, index):
        self.handle = _current_handle(index)

    @staticmethod
    def empty_like(t):
        return torch.empty_like(t, memory_format=torch.contiguous_format)

    @staticmethod
    def empty(shape, dtype, device):
        return torch.empty(shape, dtype=dtype, device=device)


def _on(device, stream, *inputs):
    return _Current(device.index) if stream is None else _On(device, stream, inputs)


# A tensor written in place, as autograd's checks of saved tensors know it.
_written = torch.autograd.graph.increment_version


def _check_out(out, x):
    _check_like("out", out, x)
    if out.requires_grad:
        _refuse("out must not require gradients")


# ------------------------------------------------------------------ gated recurrence

class ScanSaved(NamedTuple):
    """What gated_scan_backward needs of a forward."""
    x: torch.Tensor
    gate: torch.Tensor
    mask: Optional[torch.Tensor]
    states: torch.Tensor
    config: object
    has_initial_state: bool


def _scan_args(x, gate, mask, gate_normalizer, tied, dims):
    _check_x("x", x, dims)
    _check_like("gate", gate, x)
    shape = x.shape
    if shape[-1] == 0:
        _refuse("x has no channels")
    if mask is not None:
        _check_mask(mask, shape[:-1], x.device)
    if type(gate_normalizer) is not float:
        gate_normalizer = _number("gate_normalizer", gate_normalizer)
    return _scan_config(x.get_device(), x.dtype, shape[-1], True if tied else False, gate_normalizer), shape


def _scan_forward(x, gate, mask, initial_state, gate_normalizer, tied, save, out, stream):
    cfg, (B, L, D) = _scan_args(x, gate, mask, gate_normalizer, tied, 3)
    if initial_state is not None:
        _check_f32("initial_state", initial_state, (B, D), x.device)
    on = _on(x.device, stream, x, gate, mask, initial_state, out)
    own = out is None
    if own:
        out = on.empty_like(x)
    else:
        _check_out(out, x)
    last = on.empty((B, D), torch.float32, x.device)
    states = on.empty((B, -(-L // _saved_rows(x.dtype)), D), torch.float32, x.device) if save else None
    _lib.check(_lib.load().msgla_scan_forward(cfg, B, L, _rows3("x", x), _rows3("gate", gate), _ptr(mask),
                                              _ptr(initial_state), _rows3("out", out), last.data_ptr(), _ptr(states),
                                              on.handle))
    if not own:
        _written(out)
    saved = ScanSaved(x, gate, mask, states, cfg, initial_state is not None) if save else None
    return out, last, saved


def gated_scan_forward(x, gate, *, mask=None, initial_state=None, gate_normalizer: float = 16.0, tied: bool = False,
                       out=None, stream=None):
    """gated_scan without autograd: (h, last_state, saved), `saved` for gated_scan_backward.
    x and gate must not change before the backward has run."""
    return _scan_forward(x, gate, mask, initial_state, gate_normalizer, tied, True, out, stream)


def gated_scan_backward(dh, dlast, saved: ScanSaved, *, stream=None):
    """Gradients (dx, dgate, dinitial_state) of gated_scan_forward from those of h
    [B, L, D] and of the last state float32 [B, D]; either may be None (zeros).
    dinitial_state is None where the forward had no initial state."""
    x, gate, mask, states, cfg, has_state = saved
    B, L, D = x.shape
    if dh is not None:
        _check_like("dh", dh, x)
    if dlast is not None:
        _check_f32("dlast", dlast, (B, D), x.device)
    on = _on(x.device, stream, x, gate, mask, states, dh, dlast)
    dx, dgate = on.empty_like(x), on.empty_like(x)
    dstate = on.empty((B, D), torch.float32, x.device) if has_state else None
    _lib.check(_lib.load().msgla_scan_backward(cfg, B, L, _rows3("x", x), _rows3("gate", gate), _ptr(mask),
                                               states.data_ptr(), None if dh is None else _rows3("dh", dh),
                                               _ptr(dlast), _rows3("dx", dx), _rows3("dgate", dgate), _ptr(dstate),
                                               on.handle))
    return dx, dgate, dstate


def _refuse_foreign_leaves(name: str, *tensors):
    """While a graph is captured: refuses a leaf whose gradient node another, living graph made.

    The node of a leaf belongs to the stream it was made on and lives as long as a graph that
    holds it. A mark left on the node outlives the handle that left it only if such a graph exists."""
    for t in tensors:
        if t is None or not t.requires_grad or t.grad_fn is not None:
            continue
        stream = _current_handle(t.device.index)
        node = torch.autograd.graph.get_gradient_edge(t).node
        seen = node.metadata.get("msgla_stream")
        node.metadata["msgla_probe"] = True
        del node
        node = torch.autograd.graph.get_gradient_edge(t).node
        alive = node.metadata.pop("msgla_probe", False)
        if alive and seen != stream:
            _refuse(f"{name}: a tensor that requires gradients is part of a living graph made on another stream; "
                    "a backward pass captured now would break: drop that graph's outputs before the capture, or "
                    "capture the explicit forward and backward", -2)
        node.metadata["msgla_stream"] = stream
        yield node  # keeps the mark until the graph itself holds the node


class _GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, initial_state, mask, gate_normalizer, tied):
        h, last, saved = _scan_forward(x, gate, mask, initial_state, gate_normalizer, tied, True, None, None)
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(x, gate, mask, saved.states)
        ctx.rest = saved.config, saved.has_initial_state
        return h, last

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh, dlast):
        x, gate, mask, states = ctx.saved_tensors
        if dh is not None and dh.stride(-1) != 1 and dh.shape[-1] > 1:
            dh = dh.contiguous()
        if dlast is not None:
            dlast = dlast.contiguous()
        dx, dgate, dstate = gated_scan_backward(dh, dlast, ScanSaved(x, gate, mask, states, *ctx.rest))
        return dx, dgate, dstate, None, None, None


def gated_scan(x, gate, *, mask=None, initial_state=None, gate_normalizer: float = 16.0, tied: bool = False,
               out=None, stream=None):
    """The gated recurrence: (h [B, L, D], last_state float32 [B, D]).

    x, gate         [B, L, D], B up to 65535, L up to 2 ** 30; gate holds logits: a_t = sigmoid(gate_t) ** (1 / gate_normalizer).
                    A logit of -inf empties a finite state before its token (an infinite one: NaN).
    mask            optional valid tokens [B, L] (bool or uint8, nonzero = valid): a padded token
                    leaves the state as it is, its output is zero and its row is not read.
    initial_state   optional float32 [B, D] (default zeros); pass a call's last_state to go on.
    gate_normalizer a number from 2 ** -10 to 2 ** 20.
    tied            the input enters as (1 - a_t) x_t instead of x_t.
    out, stream     optional tensor for h, optional stream (neither with gradients).
    """
    if _dual_level():
        _refuse_tangents("gated_scan", x, gate, initial_state)
    if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad for t in (x, gate, initial_state)):
        if out is not None or stream is not None:
            _refuse("out and stream cannot be combined with gradients: use torch.cuda.stream(..) around both passes")
        keep = (list(_refuse_foreign_leaves("gated_scan", x, gate, initial_state))
                if torch.cuda.is_current_stream_capturing() else None)
        r = _GatedScan.apply(x, gate, initial_state, mask, gate_normalizer, tied)
        del keep
        return r
    return _scan_forward(x, gate, mask, initial_state, gate_normalizer, tied, False, out, stream)[:2]


def gated_scan_step(x, gate, state, *, mask=None, gate_normalizer: float = 16.0, tied: bool = False, out=None,
                    stream=None):
    """One token of every sequence: returns h [B, D] and updates `state` (float32 [B, D])
    in place. x, gate [B, D]; mask optional [B]: where it is zero the state stays and h is
    zero. No gradients: use gated_scan for training."""
    cfg, shape = _scan_args(x, gate, mask, gate_normalizer, tied, 2)
    _check_f32("state", state, shape, x.device)
    if _dual_level():
        _refuse_tangents("gated_scan_step", x, gate, state)
    if torch.is_grad_enabled() and (x.requires_grad or gate.requires_grad or state.requires_grad):
        _refuse("gated_scan_step has no gradients: call it under torch.no_grad()", -2)
    on = _Current(x.get_device()) if stream is None else _On(x.device, stream, (x, gate, mask, state, out))
    own = out is None
    if own:
        out = on.empty_like(x)
    else:
        _check_out(out, x)
    status = _lib.load().msgla_scan_step(cfg, shape[0], _rows2("x", x), _rows2("gate", gate),
                                         None if mask is None else mask.data_ptr(), state.data_ptr(), _rows2("out", out),
                                         on.handle)
    if status:
        _lib.check(status)
    _written(state if own else (state, out))
    return out


# ------------------------------------------------------------------ group normalisation

class NormSaved(NamedTuple):
    """What group_norm_backward needs of a forward."""
    x: torch.Tensor
    gate: Optional[torch.Tensor]
    weight: Optional[torch.Tensor]
    bias: Optional[torch.Tensor]
    mask: Optional[torch.Tensor]
    stats: torch.Tensor
    config: object


def _rows(name: str, t):
    return _rows2(name, t) if t.dim() == 2 else _rows3(name, t)


def _norm_forward(x, groups, weight, bias, gate, mask, activation, eps, center, save, out, stream):
    _check_x("x", x, 2 if isinstance(x, torch.Tensor) and x.dim() == 2 else 3)
    C = x.shape[-1]
    if not isinstance(groups, int) or groups < 1 or C == 0 or C % groups:
        _refuse(f"groups={groups} must be a positive divisor of the {C} channels")
    if not (activation is None or isinstance(activation, str)) or activation not in _ACTIVATIONS:
        _refuse(f"activation {activation!r}: none, silu or sigmoid", -2)
    if gate is not None:
        _check_like("gate", gate, x)
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            _check_f32(name, t, (C,), x.device)
    if mask is not None:
        _check_mask(mask, x.shape[:-1], x.device)
    cfg = _norm_config(x.device.index, x.dtype, C, groups, activation, bool(center), _number("eps", eps))
    N, S = x.shape[0], 1 if x.dim() == 2 else x.shape[1]
    on = _on(x.device, stream, x, weight, bias, gate, mask, out)
    own = out is None
    if own:
        out = on.empty_like(x)
    else:
        _check_out(out, x)
    stats = on.empty((N, groups, 2), torch.float32, x.device) if save else None
    ws, nbytes = _norm_workspace(cfg, N, S, False, on, x.device)
    _lib.check(_lib.load().msgla_group_norm_forward(
        cfg, N, S, _rows("x", x), None if gate is None else _rows("gate", gate), _ptr(weight), _ptr(bias), _ptr(mask),
        _rows("out", out), _ptr(stats), _ptr(ws), nbytes, on.handle))
    if not own:
        _written(out)
    return out, (NormSaved(x, gate, weight, bias, mask, stats, cfg) if save else None)


@functools.lru_cache(maxsize=1024)
def _norm_workspace_bytes(dtype: int, C: int, groups: int, N: int, S: int, gradients: int, device: int):
    n = ctypes.c_size_t()
    cfg = _lib.NormConfig(device, dtype, C, groups, 0, 1, 1.0)
    _lib.check(_lib.load().msgla_group_norm_workspace_size(cfg, N, S, gradients, ctypes.byref(n)))
    return n.value


def _norm_workspace(cfg, N, S, gradients, on, device):
    n = _norm_workspace_bytes(cfg.dtype, cfg.C, cfg.groups, N, S, 1 if gradients else 0, cfg.device)
    return (on.empty((n,), torch.uint8, device) if n else None), n


def group_norm_forward(x, groups: int, weight=None, bias=None, *, gate=None, mask=None, activation="none",
                       eps: float = 1e-5, center: bool = True, out=None, stream=None):
    """group_norm without autograd: (y, saved), `saved` for group_norm_backward. x, gate,
    weight and bias must not change before the backward has run."""
    return _norm_forward(x, groups, weight, bias, gate, mask, activation, eps, center, True, out, stream)


def group_norm_backward(dy, saved: NormSaved, *, stream=None):
    """Gradients (dx, dweight, dbias, dgate) of group_norm_forward from that of y; those
    of weight, bias and gate are None where the forward had none."""
    x, gate, weight, bias, mask, stats, cfg = saved
    _check_like("dy", dy, x)
    N, S = x.shape[0], 1 if x.dim() == 2 else x.shape[1]
    on = _on(x.device, stream, x, gate, weight, bias, mask, stats, dy)
    dx = on.empty_like(x)
    dgate = None if gate is None else on.empty_like(x)
    dw = None if weight is None else on.empty((cfg.C,), torch.float32, x.device)
    db = None if bias is None else on.empty((cfg.C,), torch.float32, x.device)
    ws, nbytes = _norm_workspace(cfg, N, S, True, on, x.device)
    _lib.check(_lib.load().msgla_group_norm_backward(
        cfg, N, S, _rows("x", x), None if gate is None else _rows("gate", gate), _ptr(weight), _ptr(bias), _ptr(mask),
        stats.data_ptr(), _rows("dy", dy), _rows("dx", dx), None if gate is None else _rows("dgate", dgate), _ptr(dw),
        _ptr(db), _ptr(ws), nbytes, on.handle))
    return dx, dw, db, dgate


class _GroupNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, gate, mask, groups, activation, eps, center):
        y, saved = _norm_forward(x, groups, weight, bias, gate, mask, activation, eps, center, True, None, None)
        ctx.save_for_backward(x, gate, weight, bias, mask, saved.stats)
        ctx.config = saved.config
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        if dy.stride(-1) != 1 and dy.shape[-1] > 1:
            dy = dy.contiguous()
        dx, dw, db, dgate = group_norm_backward(dy, NormSaved(*ctx.saved_tensors, ctx.config))
        return dx, dw, db, dgate, None, None, None, None, None


def group_norm(x, groups: int, weight=None, bias=None, *, gate=None, mask=None, activation="none", eps: float = 1e-5,
               center: bool = True, out=None, stream=None):
    """Group normalisation, channels last, with an activation or an output gate.

    x               [N, C]: every row by itself (the heads of a token, a group a head), or
                    [N, S, C]: statistics over the S rows of a sample and a group's channels.
    groups          groups of neighbouring channels; divides C.
    weight, bias    optional float32 [C].
    gate            optional, like x: y = v * act(gate) instead of y = act(v).
    mask            optional valid rows, x.shape[:-1] (bool or uint8, nonzero = valid): padded rows
                    enter no statistic, give zeros and are not read.
    activation      "none", "silu" or "sigmoid".
    center          False: divide by the root mean square, without taking the mean off.
    out, stream     optional tensor for y, optional stream (neither with gradients).
    """
    if _dual_level():
        _refuse_tangents("group_norm", x, weight, bias, gate)
    if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad for t in (x, weight, bias, gate)):
        if out is not None or stream is not None:
            _refuse("out and stream cannot be combined with gradients: use torch.cuda.stream(..) around both passes")
        keep = (list(_refuse_foreign_leaves("group_norm", x, weight, bias, gate))
                if torch.cuda.is_current_stream_capturing() else None)
        r = _GroupNorm.apply(x, weight, bias, gate, mask, groups, activation, eps, center)
        del keep
        return r
    return _norm_forward(x, groups, weight, bias, gate, mask, activation, eps, center, False, out, stream)[0]
