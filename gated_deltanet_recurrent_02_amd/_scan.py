"""ctypes binding of include/gdn_scan.h: a gated linear recurrence with one value of state for each
channel, and its gradients.

As in the rest of the package every function takes torch tensors on a HIP device, checks types,
shapes and strides, and passes raw pointers plus torch's current stream of that device to the C ABI;
outputs and workspaces that are not given are allocated from torch on that stream. x, a, b, d_o and o
may have any strides as long as the last dimension is dense. There is no autograd here: a training loop
calls the backward function itself.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from ._binding import _ACT, _DTYPE_CODE, _need, lib
from ._linear import _call, _fits, _ptr, _same_device, _size, _workspace

# Every symbol include/gdn_scan.h declares.
SCAN_EXPORTS = ("gdn_gated_scan_decode_step", "gdn_gated_scan_prefill_workspace_size", "gdn_gated_scan_prefill",
                "gdn_gated_scan_backward_workspace_size", "gdn_gated_scan_backward")

# Tokens from one kept state (`checkpoints`) to the next.
GATED_SCAN_CHECKPOINT = 64

_declared = None
_F32, _I32 = (torch.float32,), (torch.int32,)
_DENSE = torch.contiguous_format
_pack2 = struct.Struct("2q").pack


def _lib():
    global _declared
    L = lib()
    if _declared is not L:
        P, i64, i32, i = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
        n, pn = ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)
        inputs = [i64, i32, i32, P, P, P, P, P, P, i, P, P]
        for name, args in (
                ("gdn_gated_scan_decode_step", [*inputs, P, i, P, P, P]),
                ("gdn_gated_scan_prefill_workspace_size", [i64, i32, i32, pn]),
                ("gdn_gated_scan_prefill", [*inputs, P, i, P, P, P, P, n, P]),
                ("gdn_gated_scan_backward_workspace_size", [i64, i32, i32, pn]),
                ("gdn_gated_scan_backward", [*inputs, P, P, P, P, P, i, P, P, P, P, P, P, P, P, P, n, P])):
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, i
        _declared = L
    return L


def _rows(t):
    """Pointer and strides of a [B, T, C] tensor (or None) for the C ABI."""
    if t is None:
        return None, None
    return t.data_ptr(), None if t.is_contiguous() else _pack2(*t.stride()[:2])


def _is_rows(t, dt, shape, index) -> bool:
    return (t.dtype is dt and t.shape == shape and t.get_device() == index
            and (t.stride(-1) == 1 or shape[-1] == 1 or t.numel() == 0))


def _need_rows(t, name: str, dt, shape, dev) -> None:
    """The specific message for a tensor that _is_rows refuses."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a HIP device")
    if t.dtype is not dt:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dt}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    raise ValueError(f"{name} must be dense in its last dimension")


def _inputs(x, a, b, rate, lengths, name, like):
    """Sizes and the device's index of a call. `like` (called `name`): a tensor of x's shape and type, or None. The
    common path is one combined test; the specific message is found when it fails."""
    if not (isinstance(x, torch.Tensor) and x.dim() == 3):
        raise ValueError("x must be a tensor [B, T, C]")
    shape, dt, index = x.shape, x.dtype, x.get_device()
    B, T, C = shape
    try:
        if (index >= 0 and dt in _ACT and _is_rows(x, dt, shape, index) and _is_rows(a, dt, shape, index)
                and (b is None or _is_rows(b, dt, shape, index))
                and (like is None or _is_rows(like, dt, shape, index))
                and (rate is None or (rate.dtype is torch.float32 and rate.shape == (C,) and rate.get_device() == index
                                      and rate.is_contiguous()))
                and (lengths is None or (lengths.dtype is torch.int32 and lengths.shape == (B,)
                                         and lengths.get_device() == index and lengths.is_contiguous()))):
            return B, T, C, index
    except AttributeError:
        pass
    if not x.is_cuda:
        raise ValueError("x must be on a HIP device")
    if dt not in _ACT:
        raise TypeError(f"x has dtype {dt}, expected one of {_ACT}")
    dev = x.device
    for n, t in (("x", x), ("a", a), ("b", b), (name, like)):
        if t is None and n != "a":
            continue
        if not isinstance(t, torch.Tensor) or not _is_rows(t, dt, shape, index):
            _need_rows(t, n, dt, shape, dev)
    if rate is not None:
        _need(rate, "rate", (C,), _F32)
    if lengths is not None:
        _need(lengths, "lengths", (B,), _I32)
    _same_device(dev, rate=rate, lengths=lengths)
    raise ValueError("unsupported arguments")


def _state(t, name: str, shape: tuple, index: int) -> None:
    if not (isinstance(t, torch.Tensor) and t.dtype in _ACT and t.shape == shape and t.get_device() == index
            and t.is_contiguous()):
        _need(t, name, shape, _ACT)
        raise ValueError(f"{name} is on {t.device}, expected device {index}")


def _checkpoints(t, B: int, T: int, C: int, index: int) -> None:
    shape = (B, -(-T // GATED_SCAN_CHECKPOINT), C)
    if t is not None and not _fits(t, torch.float32, shape, index):
        _need(t, "checkpoints", shape, _F32)
        raise ValueError(f"checkpoints is on {t.device}, expected device {index}")


def gated_scan_decode_step(x, a, b, state, rate=None, o=None, lengths=None):
    """gdn_gated_scan_decode_step on torch tensors: T tokens of h <- alpha h + beta x with
    alpha = exp(-rate softplus(a)) and beta = sigmoid(b); updates `state` in place and returns o, the
    states after every token.

    x, a, b [B,T,C] share one dtype (fp32, bf16 or fp16); b=None: beta = 1 - alpha; rate fp32 [C] (None: 1);
    state fp32, bf16 or fp16 [B,C]; o (optional) like x; lengths (optional) int32 [B]: tokens of each
    sequence (rows of o past them are zeros)."""
    B, T, C, index = _inputs(x, a, b, rate, lengths, "o", o)
    _state(state, "state", (B, C), index)
    if o is None:
        o = torch.empty_like(x, memory_format=_DENSE)
    _call(index, _lib().gdn_gated_scan_decode_step, B, T, C, *_rows(x), *_rows(a), *_rows(b), _DTYPE_CODE[x.dtype],
          _ptr(rate), _ptr(lengths), state.data_ptr(), _DTYPE_CODE[state.dtype], *_rows(o))
    return o


def gated_scan_prefill_workspace_size(B: int, T: int, C: int) -> int:
    """gdn_gated_scan_prefill_workspace_size: bytes of workspace gated_scan_prefill needs (may be 0)."""
    return _size(_lib().gdn_gated_scan_prefill_workspace_size, B, T, C)


def gated_scan_prefill(x, a, b, state, rate=None, o=None, lengths=None, checkpoints=None, workspace=None):
    """gdn_gated_scan_prefill on torch tensors: the arguments and result of gated_scan_decode_step, for prompts.

    checkpoints (optional) fp32 [B, ceil(T / GATED_SCAN_CHECKPOINT), C] takes the states before every 64th
    token, for gated_scan_backward. `workspace` (optional) is a device buffer of at least
    gated_scan_prefill_workspace_size(...) bytes; one is allocated when omitted."""
    B, T, C, index = _inputs(x, a, b, rate, lengths, "o", o)
    _state(state, "state", (B, C), index)
    _checkpoints(checkpoints, B, T, C, index)
    if o is None:
        o = torch.empty_like(x, memory_format=_DENSE)
    need = 0 if workspace is not None else gated_scan_prefill_workspace_size(B, T, C)
    workspace, nbytes = _workspace(workspace, need, x.device)
    _call(index, _lib().gdn_gated_scan_prefill, B, T, C, *_rows(x), *_rows(a), *_rows(b), _DTYPE_CODE[x.dtype],
          _ptr(rate), _ptr(lengths), state.data_ptr(), _DTYPE_CODE[state.dtype], *_rows(o), _ptr(checkpoints),
          _ptr(workspace), nbytes)
    return o


def gated_scan_backward_workspace_size(B: int, T: int, C: int) -> int:
    """gdn_gated_scan_backward_workspace_size: bytes of workspace gated_scan_backward needs."""
    return _size(_lib().gdn_gated_scan_backward_workspace_size, B, T, C)


def gated_scan_backward(x, a, b, d_o, state0=None, dstate=None, rate=None, lengths=None, checkpoints=None,
                        state_grad: bool = False, rate_grad: bool = False, dx=None, da=None, db=None, workspace=None):
    """gdn_gated_scan_backward on torch tensors: the gradients of gated_scan_prefill (or gated_scan_decode_step)
    from d_o [B,T,C], the gradient of o, and dstate, that of the state after the call.

    x, a, b, rate, lengths as in the forward call; state0 [B,C] the state before it (None: zeros), or
    checkpoints as gated_scan_prefill wrote them, which saves making the states again; dstate [B,C] (None: zeros).
    Returns (dx, da, db, dstate0, drate); db is None without b; dstate0 (in the states' dtype, fp32 if
    none was given) and drate (fp32 [C]) are None unless state_grad / rate_grad ask for them. dx, da and db
    (optional) take the gradients, for instance as parts of one packed tensor."""
    B, T, C, index = _inputs(x, a, b, rate, lengths, "d_o", d_o)
    if d_o is None:
        raise ValueError("d_o must be a tensor [B, T, C]")
    if b is None and db is not None:
        raise ValueError("db is given without b")
    sdt = torch.float32
    if state0 is not None:
        _state(state0, "state0", (B, C), index)
        sdt = state0.dtype
    if dstate is not None:
        if state0 is not None:
            _need(dstate, "dstate", (B, C), (sdt,))
        _state(dstate, "dstate", (B, C), index)
        sdt = dstate.dtype
    _checkpoints(checkpoints, B, T, C, index)
    outs = []
    for name, t, wanted in (("dx", dx, True), ("da", da, True), ("db", db, b is not None)):
        if t is None and wanted:
            t = torch.empty_like(x, memory_format=_DENSE)
        elif t is not None and not (isinstance(t, torch.Tensor) and _is_rows(t, x.dtype, x.shape, index)):
            _need_rows(t, name, x.dtype, x.shape, x.device)
        outs.append(t)
    dx, da, db = outs
    gs = torch.empty((B, C), dtype=sdt, device=x.device) if state_grad else None
    gr = torch.empty((C,), dtype=torch.float32, device=x.device) if rate_grad else None
    need = 0 if workspace is not None else gated_scan_backward_workspace_size(B, T, C)
    workspace, nbytes = _workspace(workspace, need, x.device)
    _call(index, _lib().gdn_gated_scan_backward, B, T, C, *_rows(x), *_rows(a), *_rows(b), _DTYPE_CODE[x.dtype],
          _ptr(rate), _ptr(lengths), _ptr(state0), _ptr(checkpoints), *_rows(d_o), _ptr(dstate), _DTYPE_CODE[sdt],
          *_rows(dx), *_rows(da), *_rows(db), _ptr(gs), _ptr(gr), _ptr(workspace), nbytes)
    return dx, da, db, gs, gr
