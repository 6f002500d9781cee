"""ctypes binding of include/gdn_rotary.h: the rotation of queries and keys by their position and
their norm in every head, with the gradients, and the frequencies of common scalings.

As in the rest of the package every function takes torch tensors on a HIP device, checks types,
shapes and strides, and passes raw pointers plus torch's current stream of that device to the C ABI;
outputs and workspaces that are not given are allocated from torch on that stream. q, k, their
gradients and outputs may have any strides as long as the last dimension is dense. There is no
autograd here: a training loop calls the backward functions itself.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from ._binding import _ACT, _DTYPE_CODE, _need, lib
from ._linear import _call, _fits, _ptr, _same_device, _size, _workspace

# Every symbol include/gdn_rotary.h declares.
ROTARY_EXPORTS = ("gdn_rope", "gdn_rope_backward", "gdn_qk_norm_rope",
                  "gdn_qk_norm_rope_backward_workspace_size", "gdn_qk_norm_rope_backward")

_declared = None
_F32, _F64, _I32 = (torch.float32,), (torch.float64,), (torch.int32,)
_DENSE = torch.contiguous_format
_pack3 = struct.Struct("3q").pack


def _lib():
    global _declared
    L = lib()
    if _declared is not L:
        P, i64, i32, f32, i = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_int
        n, pn = ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)
        sizes = [i64, i32, i32, i32, i32, i32, i]
        pair, turn = [P, P, P, P], [P, P, f32, i32, P]
        weights = [P, P, i32, f32]
        for name, args in (
                ("gdn_rope", [*sizes, *pair, *turn, *pair, P]),
                ("gdn_rope_backward", [*sizes, *pair, *turn, *pair, P]),
                ("gdn_qk_norm_rope", [*sizes, *pair, *weights, *turn, *pair, P]),
                ("gdn_qk_norm_rope_backward_workspace_size", [i64, i32, i32, i32, i32, pn]),
                ("gdn_qk_norm_rope_backward", [*sizes, *pair, *pair, *weights, *turn, *pair, P, P, P, n, P])):
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, i
        _declared = L
    return L


def rope_frequencies(dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                     original_length: int | None = None, beta_fast: float = 32.0, beta_slow: float = 1.0,
                     device=None):
    """(freqs, amplitude) for `rope` and `qk_norm_rope`: the float64 tensor [dim / 2] of radians per position,
    base^(-2i/dim), and the factor of the rotated values, both as `scaling` asks for contexts `factor`
    times the trained one:

    None      unscaled
    "linear"  every frequency divided by factor
    "ntk"     base * factor^(dim / (dim - 2)): the highest frequency kept, the lowest divided by factor
    "yarn"    frequencies of more than beta_fast turns over original_length kept, of fewer than beta_slow
              divided by factor, a linear ramp over the number of turns between; amplitude 0.1 ln(factor) + 1.
              Models that ramp over the pair's index between two rounded indexes instead have other frequencies
              between the two ends: give theirs as freqs"""
    if dim < 2 or dim % 2:
        raise ValueError("dim must be even and at least 2")
    if not (base > 0 and factor >= 1):
        raise ValueError("base must be positive and factor at least 1")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if scaling == "ntk":
        if dim == 2:
            raise ValueError("ntk scaling needs dim of at least 4")
        base = base * factor ** (dim / (dim - 2))
    freqs = [base ** (-2.0 * i / dim) for i in range(dim // 2)]
    amplitude = 1.0
    if scaling == "linear":
        freqs = [f / factor for f in freqs]
    elif scaling == "yarn":
        if not original_length or original_length < 1:
            raise ValueError("yarn scaling needs original_length")
        if not beta_fast > beta_slow:
            raise ValueError("beta_fast must be larger than beta_slow")
        for i, f in enumerate(freqs):
            turns = original_length * f / (2 * math.pi)
            keep = min(max((turns - beta_slow) / (beta_fast - beta_slow), 0.0), 1.0)
            freqs[i] = keep * f + (1 - keep) * f / factor
        amplitude = 0.1 * math.log(factor) + 1.0
    return torch.tensor(freqs, dtype=torch.float64, device=device), amplitude


def _strides(t):
    """The first three strides of a [B, T, H, D] tensor for the C ABI, and whether the last is 1."""
    st = t.stride()
    return _pack3(st[0], st[1], st[2]), st[3] == 1


def _is_heads(t, dt, shape, index) -> bool:
    return (t.dtype is dt and t.shape == shape and t.get_device() == index
            and (t.is_contiguous() or t.stride(-1) == 1 or shape[-1] == 1))


def _need_heads(t, name: str, dt, shape, dev) -> None:
    """The specific message for a tensor that _is_heads refuses."""
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


def _inputs(q, k, freqs, positions, lengths, names=("q", "k"), like=None):
    """Sizes of a call, the device's index, and the strides of q and k for the C ABI (None: dense). `like`: further
    tensors, (name, tensor or None, whether q's shape and type are wanted rather than k's) each. The common path is
    one combined test; the specific message is found when it fails."""
    if not (isinstance(q, torch.Tensor) and q.dim() == 4):
        raise ValueError(f"{names[0]} must be a tensor [B, T, Hq, D]")
    if k is not None and not (isinstance(k, torch.Tensor) and k.dim() == 4):
        raise ValueError(f"{names[1]} must be a tensor [B, T, Hk, D] or None")
    qs, dt, index = q.shape, q.dtype, q.get_device()
    B, T, Hq, D = qs
    Hk, R, ks = 0, 0, None
    q_strides = k_strides = None
    try:
        good = index >= 0 and dt in _ACT
        if not q.is_contiguous():
            q_strides, dense = _strides(q)
            good = good and (dense or D == 1)
        if k is not None:
            ks = k.shape
            Hk = ks[2]
            good = (good and k.dtype is dt and k.get_device() == index and ks[0] == B and ks[1] == T and ks[3] == D)
            if not k.is_contiguous():
                k_strides, dense = _strides(k)
                good = good and (dense or D == 1)
        if freqs is not None:
            R = 2 * freqs.numel()
            good = (good and freqs.dim() == 1 and freqs.dtype is torch.float64 and freqs.get_device() == index
                    and freqs.is_contiguous())
        if positions is not None:
            good = (good and positions.dtype is torch.int32 and positions.shape == (B, T)
                    and positions.get_device() == index and positions.is_contiguous())
        if lengths is not None:
            good = (good and lengths.dtype is torch.int32 and lengths.shape == (B,) and lengths.get_device() == index
                    and lengths.is_contiguous())
        if like is not None:
            for _, t, of_q in like:
                if t is not None:
                    good = good and t.dim() == 4 and (of_q or k is not None) and _is_heads(t, dt, qs if of_q else ks, index)
        if good:
            return B, T, Hq, Hk, D, R, index, q_strides, k_strides
    except AttributeError:
        pass
    ks = (B, T, Hk, D)
    if not q.is_cuda:
        raise ValueError(f"{names[0]} must be on a HIP device")
    if dt not in _ACT:
        raise TypeError(f"{names[0]} has dtype {dt}, expected one of {_ACT}")
    dev = q.device
    if not _is_heads(q, dt, qs, index):
        _need_heads(q, names[0], dt, qs, dev)
    if k is not None and not _is_heads(k, dt, ks, index):
        _need_heads(k, names[1], dt, ks, dev)
    for n, t, of_q in like or ():
        if t is None:
            continue
        if not of_q and k is None:
            raise ValueError(f"there is no {names[1]} for {n}")
        want = qs if of_q else ks
        if not isinstance(t, torch.Tensor) or t.dim() != 4 or not _is_heads(t, dt, want, index):
            _need_heads(t, n, dt, want, dev)
    if freqs is not None:
        if not isinstance(freqs, torch.Tensor) or freqs.dim() != 1:
            raise ValueError("freqs must be a tensor [R / 2]")
        _need(freqs, "freqs", tuple(freqs.shape), _F64)
    if positions is not None:
        _need(positions, "positions", (B, T), _I32)
    if lengths is not None:
        _need(lengths, "lengths", (B,), _I32)
    _same_device(dev, freqs=freqs, positions=positions, lengths=lengths)
    raise ValueError("unsupported arguments")


def _output(t, out, strides):
    """Pointer and strides of an output like t (strides: t's, None: dense), made if it is not given, and itself."""
    if out is None:
        out = torch.empty_like(t) if strides is None else torch.empty_like(t, memory_format=_DENSE)
        return out.data_ptr(), None, out
    return out.data_ptr(), None if out.is_contiguous() else _strides(out)[0], out


def _weights(q_weight, k_weight, Hq: int, Hk: int, D: int, index: int) -> int:
    """Whether the weights have a row per head; checks them."""
    if q_weight is None and k_weight is None:
        return 0
    per_head = 1 if 2 in (getattr(q_weight, "ndim", 1), getattr(k_weight, "ndim", 1)) else 0
    for name, w, H in (("q_weight", q_weight, Hq), ("k_weight", k_weight, Hk)):
        if w is None:
            continue
        shape = (H, D) if per_head else (D,)
        if H == 0:
            raise ValueError("there is no k for k_weight")
        if not _fits(w, torch.float32, shape, index):
            _need(w, name, shape, _F32)
            raise ValueError(f"{name} is on {w.device}, expected device {index}")
    return per_head


def rope(q, k, freqs, positions=None, interleaved: bool = False, amplitude: float = 1.0, lengths=None, q_out=None,
         k_out=None):
    """gdn_rope on torch tensors: the first R = 2 len(freqs) values of every head of q [B,T,Hq,D] and k
    [B,T,Hk,D] (None: q alone) turned by their token's position; returns (q_out, k_out).

    q and k share one dtype (fp32, bf16 or fp16); freqs float64 [R/2], radians per position (see
    rope_frequencies); positions int32 [B,T] (None: 0, 1, ...); pairs are (i, i + R/2), or (2i, 2i + 1) with
    interleaved; the turned values are multiplied by amplitude; lengths (optional) int32 [B]: rows past
    them are zeros. q_out and k_out (optional) like q and k; q and k themselves work in place."""
    return _rope("gdn_rope", ("q", "k"), q, k, freqs, positions, interleaved, amplitude, lengths, q_out, k_out)


def rope_backward(dq, dk, freqs, positions=None, interleaved: bool = False, amplitude: float = 1.0, lengths=None,
                  q_out=None, k_out=None):
    """gdn_rope_backward on torch tensors: the gradients of rope's q and k from those of its results (the
    transposed rotation), with rope's other arguments."""
    return _rope("gdn_rope_backward", ("dq", "dk"), dq, dk, freqs, positions, interleaved, amplitude, lengths, q_out,
                 k_out)


def _rope(fn, names, q, k, freqs, positions, interleaved, amplitude, lengths, q_out, k_out):
    if freqs is None:
        raise ValueError("freqs must be a tensor [R / 2]")
    like = None if q_out is None and k_out is None else (("q_out", q_out, True), ("k_out", k_out, False))
    B, T, Hq, Hk, D, R, index, qs, ks = _inputs(q, k, freqs, positions, lengths, names, like)
    qp, qos, q_out = _output(q, q_out, qs)
    kp, kos, k_out = (None, None, None) if k is None else _output(k, k_out, ks)
    _call(index, getattr(_lib(), fn), B, T, Hq, Hk, D, R, _DTYPE_CODE[q.dtype], q.data_ptr(), qs, _ptr(k), ks,
          _ptr(positions), freqs.data_ptr(), amplitude, 1 if interleaved else 0, _ptr(lengths), qp, qos, kp, kos)
    return q_out, k_out


def qk_norm_rope(q, k, freqs=None, positions=None, interleaved: bool = False, amplitude: float = 1.0, lengths=None,
                 q_weight=None, k_weight=None, eps: float = 1e-6, q_out=None, k_out=None):
    """gdn_qk_norm_rope on torch tensors: every head of q and k divided by sqrt(mean x^2 + eps), times a
    weight, then turned as by `rope` (freqs=None: the norm alone); returns (q_out, k_out).

    q_weight and k_weight fp32 [D], or [Hq,D] and [Hk,D], or None (1). Unit length, as decode_step and
    prefill want their q and k, is a weight of D^-1/2. The rest as for `rope`."""
    like = None if q_out is None and k_out is None else (("q_out", q_out, True), ("k_out", k_out, False))
    B, T, Hq, Hk, D, R, index, qs, ks = _inputs(q, k, freqs, positions, lengths, like=like)
    per_head = _weights(q_weight, k_weight, Hq, Hk, D, index)
    qp, qos, q_out = _output(q, q_out, qs)
    kp, kos, k_out = (None, None, None) if k is None else _output(k, k_out, ks)
    _call(index, _lib().gdn_qk_norm_rope, B, T, Hq, Hk, D, R, _DTYPE_CODE[q.dtype], q.data_ptr(), qs, _ptr(k), ks,
          _ptr(q_weight), _ptr(k_weight), per_head, eps, _ptr(positions), _ptr(freqs), amplitude,
          1 if interleaved else 0, _ptr(lengths), qp, qos, kp, kos)
    return q_out, k_out


def qk_norm_rope_backward_workspace_size(B: int, T: int, Hq: int, Hk: int, D: int) -> int:
    """gdn_qk_norm_rope_backward_workspace_size: bytes of workspace qk_norm_rope_backward needs."""
    return _size(_lib().gdn_qk_norm_rope_backward_workspace_size, B, T, Hq, Hk, D)


def qk_norm_rope_backward(dq, dk, q, k, freqs=None, positions=None, interleaved: bool = False,
                          amplitude: float = 1.0, lengths=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                          params: bool | None = None, q_out=None, k_out=None, workspace=None):
    """gdn_qk_norm_rope_backward on torch tensors: returns (dq_in, dk_in, dq_weight, dk_weight), the gradients
    of qk_norm_rope's q, k and weights, from dq and dk, those of its results, and its arguments.

    The weights' gradients are fp32 in the weights' shape ([D] without one); params=False leaves them
    out (None), and a weight of None has none unless params=True asks for it. q_out and k_out (optional) take
    dq_in and dk_in; dq and dk themselves work in place."""
    if not (isinstance(dq, torch.Tensor) and dq.dim() == 4):
        raise ValueError("dq must be a tensor [B, T, Hq, D]")
    if (k is None) != (dk is None):
        raise ValueError("k and dk are given together or not at all")
    B, T, Hq, Hk, D, R, index, qs, ks = _inputs(
        q, k, freqs, positions, lengths,
        like=(("dq", dq, True), ("dk", dk, False), ("q_out", q_out, True), ("k_out", k_out, False)))
    per_head = _weights(q_weight, k_weight, Hq, Hk, D, index)
    qp, qos, q_out = _output(q, q_out, qs)
    kp, kos, k_out = (None, None, None) if k is None else _output(k, k_out, ks)
    gqs = None if dq.is_contiguous() else _strides(dq)[0]
    gks = None if dk is None or dk.is_contiguous() else _strides(dk)[0]
    grads = []
    for w, H in ((q_weight, Hq), (k_weight, Hk)):
        want = H > 0 and (w is not None if params is None else params)
        if want and w is not None:
            grads.append(torch.empty_like(w))
        else:
            shape = (H, D) if per_head else (D,)
            grads.append(torch.empty(shape, dtype=torch.float32, device=q.device) if want else None)
    wanted = grads[0] is not None or grads[1] is not None
    need = qk_norm_rope_backward_workspace_size(B, T, Hq, Hk, D) if wanted and workspace is None else 0
    workspace, nbytes = _workspace(workspace, need, q.device)
    _call(index, _lib().gdn_qk_norm_rope_backward, B, T, Hq, Hk, D, R, _DTYPE_CODE[q.dtype], dq.data_ptr(), gqs, _ptr(dk),
          gks, q.data_ptr(), qs, _ptr(k), ks, _ptr(q_weight), _ptr(k_weight), per_head, eps, _ptr(positions),
          _ptr(freqs), amplitude, 1 if interleaved else 0, _ptr(lengths), qp, qos, kp, kos, _ptr(grads[0]),
          _ptr(grads[1]), _ptr(workspace), nbytes)
    return q_out, k_out, grads[0], grads[1]
