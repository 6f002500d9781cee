"""ctypes binding of include/gdn_linear.h: linear attention with a decay for each head, its
gradients, and layer norm.

As in the rest of the package every function takes torch tensors on a HIP device, checks types,
shapes and contiguity, and passes raw pointers plus torch's current stream of that device to the
C ABI; outputs and workspaces that are not given are allocated from torch on that stream. There
is no autograd here: a training loop calls the backward functions itself.
"""
from __future__ import annotations

import ctypes

import torch

from ._binding import _ACT, _DTYPE_CODE, _need, _ptr, _stream, check, lib

# Every symbol include/gdn_linear.h declares.
LINEAR_EXPORTS = ("gdn_linear_attn_decode_step", "gdn_linear_attn_prefill_workspace_size",
                  "gdn_linear_attn_prefill", "gdn_linear_attn_backward_workspace_size",
                  "gdn_linear_attn_backward", "gdn_layer_norm",
                  "gdn_layer_norm_backward_workspace_size", "gdn_layer_norm_backward")

_declared = None
_F32 = (torch.float32,)
_I32 = (torch.int32,)


def _lib():
    global _declared
    L = lib()
    if _declared is not L:
        P, i64, i32, f32, i = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_int
        n, pn = ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)
        attn = [i64, i32, i32, i32, i32, i32, P, P, P, i, P, P]
        for name, args in (
                ("gdn_linear_attn_decode_step", [*attn, P, i, P, f32, P]),
                ("gdn_linear_attn_prefill_workspace_size", [i64, i32, i32, i32, i32, pn]),
                ("gdn_linear_attn_prefill", [*attn, P, i, P, f32, P, n, P]),
                ("gdn_linear_attn_backward_workspace_size", [i64, i32, i32, i32, i32, i32, pn]),
                ("gdn_linear_attn_backward", [*attn, P, P, P, i, P, P, P, P, P, f32, P, n, P]),
                ("gdn_layer_norm", [i64, i32, i32, P, i, P, P, P, P, P, f32, P]),
                ("gdn_layer_norm_backward_workspace_size", [i64, i32, i32, pn]),
                ("gdn_layer_norm_backward", [i64, i32, i32, P, P, i, P, P, P, P, P, P, P, n, P])):
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, i
        _declared = L
    return L


def _call(dev: torch.device, fn, *args) -> None:
    """One call of the C ABI with `dev` as the current device and its current stream."""
    if dev.index == torch.cuda.current_device():
        check(fn(*args, _stream(dev)))
    else:
        with torch.cuda.device(dev):
            check(fn(*args, _stream(dev)))


def _same_device(dev: torch.device, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")


def _workspace(workspace, need: int, dev: torch.device):
    """The given workspace (checked) or one of `need` bytes: (tensor or None, bytes)."""
    if workspace is None:
        return (torch.empty(need, dtype=torch.uint8, device=dev), need) if need else (None, 0)
    if not (isinstance(workspace, torch.Tensor) and workspace.is_cuda and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous device tensor")
    _same_device(dev, workspace=workspace)
    return workspace, workspace.numel() * workspace.element_size()


def _size(fn, *args) -> int:
    n = ctypes.c_size_t(0)
    check(fn(*args, ctypes.byref(n)))
    return n.value


def _attn_inputs(q, k, v, decay, lengths):
    if not (isinstance(q, torch.Tensor) and q.dim() == 4):
        raise ValueError("q must be a tensor [B, T, Hk, dk]")
    if not (isinstance(v, torch.Tensor) and v.dim() == 4):
        raise ValueError("v must be a tensor [B, T, H, dv]")
    B, T, Hk, dk = q.shape
    H, dv = v.shape[2:]
    _need(q, "q", (B, T, Hk, dk), _ACT)
    _need(k, "k", (B, T, Hk, dk), (q.dtype,))
    _need(v, "v", (B, T, H, dv), (q.dtype,))
    _need(decay, "decay", (H,), _F32)
    if lengths is not None:
        _need(lengths, "lengths", (B,), _I32)
    dev = q.device
    if not (k.device == v.device == decay.device == dev and (lengths is None or lengths.device == dev)):
        _same_device(dev, k=k, v=v, decay=decay, lengths=lengths)
    return B, T, H, Hk, dk, dv


def linear_attn_decode_step(q, k, v, decay, state, o=None, scale: float = 1.0, lengths=None):
    """gdn_linear_attn_decode_step on torch tensors: T tokens of S <- decay S + v k^T,
    o = S (scale q); updates `state` in place and returns o.

    q, k [B,T,Hk,dk] and v [B,T,H,dv] share one dtype (fp32, bf16 or fp16), Hk divides H; decay
    fp32 [H]; state fp32, bf16 or fp16 [B,H,dv,dk]; o (optional) [B,T,H,dv] in the activation
    dtype; lengths (optional) int32 [B]: tokens of each sequence (rows of o past them are zeros)."""
    B, T, H, Hk, dk, dv = _attn_inputs(q, k, v, decay, lengths)
    _need(state, "state", (B, H, dv, dk), _ACT)
    if o is None:
        o = torch.empty_like(v)
    _need(o, "o", (B, T, H, dv), (q.dtype,))
    if not (state.device == o.device == q.device):
        _same_device(q.device, state=state, o=o)
    _call(q.device, _lib().gdn_linear_attn_decode_step, B, T, H, Hk, dk, dv, _ptr(q), _ptr(k), _ptr(v),
          _DTYPE_CODE[q.dtype], _ptr(decay), _ptr(lengths), _ptr(state), _DTYPE_CODE[state.dtype],
          _ptr(o), float(scale))
    return o


def linear_attn_prefill_workspace_size(B: int, T: int, H: int, dk: int, dv: int) -> int:
    """gdn_linear_attn_prefill_workspace_size: bytes of workspace linear_attn_prefill needs (may be 0)."""
    return _size(_lib().gdn_linear_attn_prefill_workspace_size, B, T, H, dk, dv)


def linear_attn_prefill(q, k, v, decay, state, o=None, scale: float = 1.0, lengths=None, workspace=None):
    """gdn_linear_attn_prefill on torch tensors: the arguments and result of
    linear_attn_decode_step, for prompts. `workspace` (optional) is a device buffer of at least
    linear_attn_prefill_workspace_size(...) bytes; one is allocated when omitted."""
    B, T, H, Hk, dk, dv = _attn_inputs(q, k, v, decay, lengths)
    _need(state, "state", (B, H, dv, dk), _ACT)
    if o is None:
        o = torch.empty_like(v)
    _need(o, "o", (B, T, H, dv), (q.dtype,))
    _same_device(q.device, state=state, o=o)
    need = 0 if workspace is not None else linear_attn_prefill_workspace_size(B, T, H, dk, dv)
    workspace, nbytes = _workspace(workspace, need, q.device)
    _call(q.device, _lib().gdn_linear_attn_prefill, B, T, H, Hk, dk, dv, _ptr(q), _ptr(k), _ptr(v),
          _DTYPE_CODE[q.dtype], _ptr(decay), _ptr(lengths), _ptr(state), _DTYPE_CODE[state.dtype],
          _ptr(o), float(scale), _ptr(workspace), nbytes)
    return o


def linear_attn_backward_workspace_size(B: int, T: int, H: int, Hk: int, dk: int, dv: int) -> int:
    """gdn_linear_attn_backward_workspace_size: bytes of workspace linear_attn_backward needs."""
    return _size(_lib().gdn_linear_attn_backward_workspace_size, B, T, H, Hk, dk, dv)


def linear_attn_backward(q, k, v, decay, d_o, state0=None, dstate=None, scale: float = 1.0, lengths=None,
                         state_grad: bool = False, decay_grad: bool = False, workspace=None):
    """gdn_linear_attn_backward on torch tensors: the gradients of linear_attn_prefill (or
    linear_attn_decode_step) from d_o [B,T,H,dv], the gradient of o, and dstate, that of the
    state after the call.

    q, k, v, decay, scale, lengths as in the forward call; state0 [B,H,dv,dk] the state before it
    (None: zeros); dstate like state0 and of its dtype (None: zeros). Returns
    (dq, dk, dv, dstate0, ddecay); dstate0 (in the states' dtype, fp32 if none was given) and
    ddecay (fp32 [H]) are None unless state_grad / decay_grad ask for them."""
    B, T, H, Hk, dk, dv = _attn_inputs(q, k, v, decay, lengths)
    _need(d_o, "d_o", (B, T, H, dv), (q.dtype,))
    sdt = torch.float32
    if state0 is not None:
        _need(state0, "state0", (B, H, dv, dk), _ACT)
        sdt = state0.dtype
    if dstate is not None:
        _need(dstate, "dstate", (B, H, dv, dk), _ACT if state0 is None else (sdt,))
        sdt = dstate.dtype
    _same_device(q.device, d_o=d_o, state0=state0, dstate=dstate)
    gq, gk, gv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    gs = torch.empty((B, H, dv, dk), dtype=sdt, device=q.device) if state_grad else None
    gd = torch.empty((H,), dtype=torch.float32, device=q.device) if decay_grad else None
    need = 0 if workspace is not None else linear_attn_backward_workspace_size(B, T, H, Hk, dk, dv)
    workspace, nbytes = _workspace(workspace, need, q.device)
    _call(q.device, _lib().gdn_linear_attn_backward, B, T, H, Hk, dk, dv, _ptr(q), _ptr(k), _ptr(v),
          _DTYPE_CODE[q.dtype], _ptr(decay), _ptr(lengths), _ptr(state0), _ptr(d_o), _ptr(dstate),
          _DTYPE_CODE[sdt], _ptr(gq), _ptr(gk), _ptr(gv), _ptr(gs), _ptr(gd), float(scale),
          _ptr(workspace), nbytes)
    return gq, gk, gv, gs, gd


def _norm_shape(x, weight, bias):
    """(rows, G, C) of a layer-norm call; weight and bias have x's last dimension, or its last two."""
    if not (isinstance(x, torch.Tensor) and x.dim() >= 1):
        raise ValueError("x must be a tensor with at least one dimension")
    C = x.shape[-1]
    shape = (C,)
    for p in (weight, bias):
        if isinstance(p, torch.Tensor) and p.dim() == 2:
            shape = tuple(x.shape[-2:])
    _need(x, "x", x.shape, _ACT)
    if weight is not None:
        _need(weight, "weight", shape, _F32)
    if bias is not None:
        _need(bias, "bias", shape, _F32)
    _same_device(x.device, weight=weight, bias=bias)
    G = shape[0] if len(shape) == 2 else 1
    return (x.numel() // C if C else 0), G, C, shape


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, stats: bool = False, y=None):
    """gdn_layer_norm on torch tensors: normalises x over its last dimension and returns y, or
    (y, mean, rstd) with stats=True, what layer_norm_backward needs.

    x [..., C] fp32, bf16 or fp16; weight and bias fp32 [C], or [G, C] with G the last but one
    dimension of x (every head its own affine), or None; y (optional) like x (x itself works in
    place); mean and rstd fp32 [...]."""
    rows, G, C, _ = _norm_shape(x, weight, bias)
    if y is None:
        y = torch.empty_like(x)
    _need(y, "y", x.shape, (x.dtype,))
    if y.device != x.device:
        _same_device(x.device, y=y)
    mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device) if stats else None
    rstd = torch.empty_like(mean) if stats else None
    _call(x.device, _lib().gdn_layer_norm, rows, G, C, _ptr(x), _DTYPE_CODE[x.dtype], _ptr(weight),
          _ptr(bias), _ptr(y), _ptr(mean), _ptr(rstd), float(eps))
    return (y, mean, rstd) if stats else y


def layer_norm_backward_workspace_size(rows: int, G: int, C: int) -> int:
    """gdn_layer_norm_backward_workspace_size: bytes of workspace layer_norm_backward needs."""
    return _size(_lib().gdn_layer_norm_backward_workspace_size, rows, G, C)


def layer_norm_backward(dy, x, mean, rstd, weight=None, params: bool | None = None, workspace=None):
    """gdn_layer_norm_backward on torch tensors: returns (dx, dweight, dbias) from dy, the gradient
    of y, and layer_norm's inputs and statistics.

    dweight and dbias are fp32 in weight's shape ([C] without one); params=False leaves them out
    (None), and so does weight=None unless params=True asks for them."""
    rows, G, C, shape = _norm_shape(x, weight, None)
    _need(dy, "dy", x.shape, (x.dtype,))
    _need(mean, "mean", x.shape[:-1], _F32)
    _need(rstd, "rstd", x.shape[:-1], _F32)
    _same_device(x.device, dy=dy, mean=mean, rstd=rstd)
    want = weight is not None if params is None else params
    dx = torch.empty_like(x)
    dw = torch.empty(shape, dtype=torch.float32, device=x.device) if want else None
    db = torch.empty(shape, dtype=torch.float32, device=x.device) if want else None
    need = layer_norm_backward_workspace_size(rows, G, C) if want and workspace is None else 0
    workspace, nbytes = _workspace(workspace, need, x.device)
    _call(x.device, _lib().gdn_layer_norm_backward, rows, G, C, _ptr(dy), _ptr(x), _DTYPE_CODE[x.dtype],
          _ptr(weight), _ptr(mean), _ptr(rstd), _ptr(dx), _ptr(dw), _ptr(db), _ptr(workspace), nbytes)
    return dx, dw, db
