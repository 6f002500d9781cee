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

from ._binding import _ACT, _DTYPE_CODE, _need, check, lib

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


# The current device's index without torch's lazy-initialisation check (a device tensor exists, so
# torch is initialised); torch builds without the raw accessors take the public ones.
_get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_get_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(index: int, fn, *args) -> None:
    """One call of the C ABI with device `index` as the current device and its current stream."""
    if index == _get_device():
        status = fn(*args, _get_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _get_stream(index))
    if status:
        check(status)


def _ptr(t):
    return None if t is None else t.data_ptr()


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


def _attn_inputs(q, k, v, decay, lengths, like_v):
    """Sizes and the device's index of a call. `like_v`: a tensor of v's shape and type. The common path is
    one combined test; the specific message is found when it fails."""
    if not (isinstance(q, torch.Tensor) and q.dim() == 4):
        raise ValueError("q must be a tensor [B, T, Hk, dk]")
    if not (isinstance(v, torch.Tensor) and v.dim() == 4):
        raise ValueError("v must be a tensor [B, T, H, dv]")
    qs, vs, dt, index = q.shape, v.shape, q.dtype, q.get_device()
    B, T, Hk, dk = qs
    H, dv = vs[2], vs[3]
    try:
        if (index >= 0 and dt in _ACT and k.dtype is dt and v.dtype is dt and like_v.dtype is dt
                and decay.dtype is torch.float32 and k.shape == qs and like_v.shape == vs and vs[0] == B
                and vs[1] == T and decay.shape == (H,) and k.get_device() == index and v.get_device() == index
                and decay.get_device() == index and like_v.get_device() == index and q.is_contiguous()
                and k.is_contiguous() and v.is_contiguous() and like_v.is_contiguous() and decay.is_contiguous()
                and (lengths is None or (lengths.dtype is torch.int32 and lengths.shape == (B,)
                                         and lengths.get_device() == index and lengths.is_contiguous()))):
            return B, T, H, Hk, dk, dv, index
    except AttributeError:
        pass
    _need(q, "q", (B, T, Hk, dk), _ACT)
    _need(k, "k", (B, T, Hk, dk), (dt,))
    _need(v, "v", (B, T, H, dv), (dt,))
    _need(decay, "decay", (H,), _F32)
    if lengths is not None:
        _need(lengths, "lengths", (B,), _I32)
    _need(like_v, "o or d_o", (B, T, H, dv), (dt,))
    _same_device(q.device, k=k, v=v, decay=decay, lengths=lengths, o_or_d_o=like_v)
    raise ValueError("unsupported arguments")


def _state(t, name: str, shape: tuple, index: int) -> None:
    if not (isinstance(t, torch.Tensor) and t.dtype in _ACT and t.shape == shape and t.get_device() == index
            and t.is_contiguous()):
        _need(t, name, shape, _ACT)
        raise ValueError(f"{name} is on {t.device}, expected device {index}")


def linear_attn_decode_step(q, k, v, decay, state, o=None, scale: float = 1.0, lengths=None):
    """gdn_linear_attn_decode_step on torch tensors: T tokens of S <- decay S + v k^T,
    o = S (scale q); updates `state` in place and returns o.

    q, k [B,T,Hk,dk] and v [B,T,H,dv] share one dtype (fp32, bf16 or fp16), Hk divides H; decay
    fp32 [H]; state fp32, bf16 or fp16 [B,H,dv,dk]; o (optional) [B,T,H,dv] in the activation
    dtype; lengths (optional) int32 [B]: tokens of each sequence (rows of o past them are zeros)."""
    if o is None:
        o = torch.empty_like(v)
    B, T, H, Hk, dk, dv, index = _attn_inputs(q, k, v, decay, lengths, o)
    _state(state, "state", (B, H, dv, dk), index)
    _call(index, _lib().gdn_linear_attn_decode_step, B, T, H, Hk, dk, dv, q.data_ptr(), k.data_ptr(),
          v.data_ptr(), _DTYPE_CODE[q.dtype], decay.data_ptr(), _ptr(lengths), state.data_ptr(),
          _DTYPE_CODE[state.dtype], o.data_ptr(), scale)
    return o


def linear_attn_prefill_workspace_size(B: int, T: int, H: int, dk: int, dv: int) -> int:
    """gdn_linear_attn_prefill_workspace_size: bytes of workspace linear_attn_prefill needs (may be 0)."""
    return _size(_lib().gdn_linear_attn_prefill_workspace_size, B, T, H, dk, dv)


def linear_attn_prefill(q, k, v, decay, state, o=None, scale: float = 1.0, lengths=None, workspace=None):
    """gdn_linear_attn_prefill on torch tensors: the arguments and result of
    linear_attn_decode_step, for prompts. `workspace` (optional) is a device buffer of at least
    linear_attn_prefill_workspace_size(...) bytes; one is allocated when omitted."""
    if o is None:
        o = torch.empty_like(v)
    B, T, H, Hk, dk, dv, index = _attn_inputs(q, k, v, decay, lengths, o)
    _state(state, "state", (B, H, dv, dk), index)
    need = 0 if workspace is not None else linear_attn_prefill_workspace_size(B, T, H, dk, dv)
    workspace, nbytes = _workspace(workspace, need, q.device)
    _call(index, _lib().gdn_linear_attn_prefill, B, T, H, Hk, dk, dv, q.data_ptr(), k.data_ptr(),
          v.data_ptr(), _DTYPE_CODE[q.dtype], decay.data_ptr(), _ptr(lengths), state.data_ptr(),
          _DTYPE_CODE[state.dtype], o.data_ptr(), scale, _ptr(workspace), nbytes)
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
    B, T, H, Hk, dk, dv, index = _attn_inputs(q, k, v, decay, lengths, d_o)
    sdt = torch.float32
    if state0 is not None:
        _state(state0, "state0", (B, H, dv, dk), index)
        sdt = state0.dtype
    if dstate is not None:
        if state0 is not None:
            _need(dstate, "dstate", (B, H, dv, dk), (sdt,))
        _state(dstate, "dstate", (B, H, dv, dk), index)
        sdt = dstate.dtype
    gq, gk, gv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    gs = torch.empty((B, H, dv, dk), dtype=sdt, device=q.device) if state_grad else None
    gd = torch.empty((H,), dtype=torch.float32, device=q.device) if decay_grad else None
    need = 0 if workspace is not None else linear_attn_backward_workspace_size(B, T, H, Hk, dk, dv)
    workspace, nbytes = _workspace(workspace, need, q.device)
    _call(index, _lib().gdn_linear_attn_backward, B, T, H, Hk, dk, dv, q.data_ptr(), k.data_ptr(),
          v.data_ptr(), _DTYPE_CODE[q.dtype], decay.data_ptr(), _ptr(lengths), _ptr(state0), d_o.data_ptr(),
          _ptr(dstate), _DTYPE_CODE[sdt], gq.data_ptr(), gk.data_ptr(), gv.data_ptr(), _ptr(gs), _ptr(gd),
          scale, _ptr(workspace), nbytes)
    return gq, gk, gv, gs, gd


def _fits(t, dtype, shape, index: int) -> bool:
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index
            and t.is_contiguous())


def _norm_shape(x, weight, bias, like_x, name="y"):
    """(rows, G, C, affine shape, device index) of a layer-norm call; weight and bias have x's last
    dimension, or its last two. `like_x`: a tensor of x's shape and type (`name`), or x itself. The common
    path is one combined test; the specific message is found when it fails."""
    if not (isinstance(x, torch.Tensor) and x.dim() >= 1):
        raise ValueError("x must be a tensor with at least one dimension")
    xs, index, dt = x.shape, x.get_device(), x.dtype
    C = xs[-1]
    two = (weight is not None and getattr(weight, "ndim", 1) == 2) or (bias is not None and getattr(bias, "ndim", 1) == 2)
    shape = xs[-2:] if two else xs[-1:]
    try:
        good = (index >= 0 and dt in _ACT and x.is_contiguous()
                and (like_x is x or (like_x.dtype is dt and like_x.shape == xs and like_x.get_device() == index
                                     and like_x.is_contiguous()))
                and (weight is None or (weight.dtype is torch.float32 and weight.shape == shape
                                        and weight.get_device() == index and weight.is_contiguous()))
                and (bias is None or (bias.dtype is torch.float32 and bias.shape == shape
                                      and bias.get_device() == index and bias.is_contiguous())))
    except AttributeError:
        good = False
    if not good:
        _need(x, "x", xs, _ACT)
        for n, p in (("weight", weight), ("bias", bias)):
            if p is not None:
                _need(p, n, tuple(shape), _F32)
        _need(like_x, name, xs, (dt,))
        _same_device(x.device, weight=weight, bias=bias, **{name: like_x})
        raise ValueError("unsupported arguments")
    return (x.numel() // C if C else 0), shape[0] if two else 1, C, shape, index


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, stats: bool = False, y=None):
    """gdn_layer_norm on torch tensors: normalises x over its last dimension and returns y, or
    (y, mean, rstd) with stats=True, what layer_norm_backward needs.

    x [..., C] fp32, bf16 or fp16; weight and bias fp32 [C], or [G, C] with G the last but one
    dimension of x (every head its own affine), or None; y (optional) like x (x itself works in
    place); mean and rstd fp32 [...]."""
    rows, G, C, _, index = _norm_shape(x, weight, bias, x if y is None else y)
    if y is None:
        y = torch.empty_like(x)
    mean = rstd = None
    if stats:
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
    _call(index, _lib().gdn_layer_norm, rows, G, C, x.data_ptr(), _DTYPE_CODE[x.dtype], _ptr(weight),
          _ptr(bias), y.data_ptr(), _ptr(mean), _ptr(rstd), eps)
    return (y, mean, rstd) if stats else y


def layer_norm_backward_workspace_size(rows: int, G: int, C: int) -> int:
    """gdn_layer_norm_backward_workspace_size: bytes of workspace layer_norm_backward needs."""
    return _size(_lib().gdn_layer_norm_backward_workspace_size, rows, G, C)


def layer_norm_backward(dy, x, mean, rstd, weight=None, params: bool | None = None, workspace=None):
    """gdn_layer_norm_backward on torch tensors: returns (dx, dweight, dbias) from dy, the gradient
    of y, and layer_norm's inputs and statistics.

    dweight and dbias are fp32 in weight's shape ([C] without one); params=False leaves them out
    (None), and so does weight=None unless params=True asks for them."""
    rows, G, C, shape, index = _norm_shape(x, weight, None, dy, "dy")
    for name, t in (("mean", mean), ("rstd", rstd)):
        if not _fits(t, torch.float32, x.shape[:-1], index):
            _need(t, name, x.shape[:-1], _F32)
            _same_device(x.device, **{name: t})
    want = weight is not None if params is None else params
    dx = torch.empty_like(x)
    dw = torch.empty(shape, dtype=torch.float32, device=x.device) if want else None
    db = torch.empty_like(dw) if want else None
    need = layer_norm_backward_workspace_size(rows, G, C) if want and workspace is None else 0
    workspace, nbytes = _workspace(workspace, need, x.device)
    _call(index, _lib().gdn_layer_norm_backward, rows, G, C, dy.data_ptr(), x.data_ptr(), _DTYPE_CODE[x.dtype],
          _ptr(weight), mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), _ptr(dw), _ptr(db), _ptr(workspace),
          nbytes)
    return dx, dw, db
