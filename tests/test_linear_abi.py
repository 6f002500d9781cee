"""The C ABI of include/gdn_linear.h on the CPU: exports, refusals of invalid arguments before any
HIP call, empty work, workspace sizes, and the binding's own checks."""
import ctypes
import os
import re

import pytest
import torch

import gated_deltanet_recurrent_02_amd as gdn
from gated_deltanet_recurrent_02_amd import _binding as bd
from gated_deltanet_recurrent_02_amd import _linear as ln

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdn_linear.h")
INVALID, UNSUPPORTED, HIP = bd.GDN_ERR_INVALID_ARGUMENT, bd.GDN_ERR_UNSUPPORTED, bd.GDN_ERR_HIP
F32, BF16 = bd.GDN_F32, bd.GDN_BF16
BASE = 0x7F0000000000  # a fake, 256-byte aligned device address
MB = 1 << 20
NULL = ctypes.c_void_p(0)

# Fake device pointers are only ever passed where no GPU is visible.
fake_ptrs = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="passes fake device pointers")


def P(off=0):
    return ctypes.c_void_p(BASE + off)


def last_error():
    return gdn.lib().gdn_last_error().decode()


def test_header_declares_the_binding_exports():
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(gdn_[a-z0-9_]+)\s*\(", text)))
    assert declared == sorted(gdn.LINEAR_EXPORTS)
    L = ctypes.CDLL(bd.LIBRARY)
    for name in declared:
        assert hasattr(L, name), name


def attn(prefill=False, B=2, T=4, H=4, Hk=2, dk=16, dv=16, q=P(0), k=P(16 * MB), v=P(32 * MB), act=F32,
         decay=P(48 * MB), lengths=P(64 * MB), state=P(80 * MB), sdt=F32, o=P(160 * MB), ws=P(1 << 40),
         wsb=1 << 40):
    L = ln._lib()
    if prefill:
        return L.gdn_linear_attn_prefill(B, T, H, Hk, dk, dv, q, k, v, act, decay, lengths, state, sdt, o, 1.0,
                                         ws, wsb, None)
    return L.gdn_linear_attn_decode_step(B, T, H, Hk, dk, dv, q, k, v, act, decay, lengths, state, sdt, o, 1.0, None)


ATTN_REFUSALS = [
    (dict(H=0), INVALID, "H must be"),
    (dict(B=-1), INVALID, "B and T"),
    (dict(T=-3), INVALID, "B and T"),
    (dict(Hk=0), INVALID, "Hk"),
    (dict(Hk=3), INVALID, "Hk"),
    (dict(Hk=8), INVALID, "Hk"),
    (dict(dk=48, dv=48), UNSUPPORTED, "head dims"),
    (dict(dk=64, dv=128), UNSUPPORTED, "head dims"),
    (dict(act=7), INVALID, "dtype"),
    (dict(sdt=-1), INVALID, "dtype"),
    (dict(q=NULL), INVALID, "q is NULL"),
    (dict(decay=NULL), INVALID, "decay is NULL"),
    (dict(state=NULL), INVALID, "state is NULL"),
    (dict(lengths=P(64 * MB + 4)), INVALID, "lengths is not 16-byte aligned"),
    (dict(o=P(160 * MB + 8)), INVALID, "o is not 16-byte aligned"),
    (dict(o=P(0)), INVALID, "o overlaps q"),
    (dict(o=P(64 * MB)), INVALID, "o overlaps lengths"),
    (dict(o=P(80 * MB + 1024)), INVALID, "o overlaps state"),
    (dict(state=P(32 * MB)), INVALID, "state overlaps v"),
    (dict(state=P(48 * MB)), INVALID, "state overlaps decay"),
    (dict(B=1 << 26, H=32, Hk=32), INVALID, "B * H"),
    (dict(B=1 << 40), INVALID, "B * H"),
    (dict(B=1 << 62, H=8), INVALID, "B * H"),
    (dict(B=1 << 20, H=1 << 5), UNSUPPORTED, "B * H * 8 * dk"),
    (dict(B=1 << 20, H=4, T=(1 << 31) - 1, dk=128, dv=128), UNSUPPORTED, "B * H * 8 * dk"),
    (dict(B=1 << 18, H=4, T=(1 << 31) - 1, dk=128, dv=128), UNSUPPORTED, "T must be"),
    (dict(T=1 << 30), UNSUPPORTED, "T must be"),
]


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("kw,status,msg", ATTN_REFUSALS)
@fake_ptrs
def test_attention_rejects(prefill, kw, status, msg):
    assert attn(prefill, **kw) == status
    assert msg in last_error() and last_error()


@fake_ptrs
def test_prefill_rejects_its_workspace():
    kw = dict(B=1, T=4096, H=1, Hk=1, dk=128, dv=128)
    n = gdn.linear_attn_prefill_workspace_size(1, 4096, 1, 128, 128)
    if n:
        assert attn(True, **kw, ws=NULL) == INVALID and "workspace is NULL" in last_error()
        assert attn(True, **kw, wsb=n - 1) == INVALID and "needed" in last_error()
        assert attn(True, **kw, ws=P(80 * MB)) == INVALID and "overlaps workspace" in last_error()
    assert attn(True, **kw, wsb=n) == HIP


@fake_ptrs
def test_attention_empty_work_and_calls_without_a_device():
    for prefill in (False, True):
        for B, T in ((0, 1), (3, 0), (0, 0)):
            assert attn(prefill, B=B, T=T, q=NULL, k=NULL, v=NULL, decay=NULL, lengths=NULL, state=NULL, o=NULL,
                        ws=NULL, wsb=0) == 0
            assert last_error() == ""
        assert attn(prefill) == HIP          # valid, but there is no device
        assert attn(prefill, lengths=NULL) == HIP
        assert attn(prefill, q=P(0), k=P(0)) == HIP   # q and k may alias


def backward(B=2, T=4, H=4, Hk=2, dk=16, dv=16, q=P(0), k=P(16 * MB), v=P(32 * MB), act=F32, decay=P(48 * MB),
             lengths=P(64 * MB), state0=P(80 * MB), d_o=P(96 * MB), dstate=P(112 * MB), sdt=F32, dq=P(128 * MB),
             gk=P(144 * MB), gv=P(160 * MB), dstate0=P(176 * MB), ddecay=P(192 * MB), ws=P(1 << 40), wsb=1 << 40):
    return ln._lib().gdn_linear_attn_backward(B, T, H, Hk, dk, dv, q, k, v, act, decay, lengths, state0, d_o, dstate,
                                              sdt, dq, gk, gv, dstate0, ddecay, 1.0, ws, wsb, None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(H=0), INVALID, "H must be"),
    (dict(Hk=3), INVALID, "Hk"),
    (dict(dk=96, dv=96), UNSUPPORTED, "head dims"),
    (dict(act=3), INVALID, "dtype"),
    (dict(sdt=3), INVALID, "dtype"),
    (dict(d_o=NULL), INVALID, "d_o is NULL"),
    (dict(dq=NULL), INVALID, "dq is NULL"),
    (dict(gk=P(144 * MB + 2)), INVALID, "dk_out is not 16-byte aligned"),
    (dict(ddecay=P(192 * MB + 4)), INVALID, "ddecay is not 16-byte aligned"),
    (dict(state0=P(80 * MB + 8)), INVALID, "state0 is not 16-byte aligned"),
    (dict(dq=P(0)), INVALID, "dq overlaps q"),
    (dict(gk=P(128 * MB)), INVALID, "dk_out overlaps dq"),
    (dict(gv=P(96 * MB)), INVALID, "dv_out overlaps d_o"),
    (dict(dstate0=P(112 * MB)), INVALID, "dstate0 overlaps dstate"),
    (dict(dstate0=P(80 * MB)), INVALID, "dstate0 overlaps state0"),
    (dict(ddecay=P(48 * MB)), INVALID, "ddecay overlaps decay"),
    (dict(ws=NULL), INVALID, "workspace is NULL"),
    (dict(wsb=0), INVALID, "needed"),
    (dict(ws=P(160 * MB)), INVALID, "workspace overlaps"),
])
@fake_ptrs
def test_backward_rejects(kw, status, msg):
    assert backward(**kw) == status
    assert msg in last_error()


@fake_ptrs
def test_backward_empty_work_and_calls_without_a_device():
    none = dict(q=NULL, k=NULL, v=NULL, d_o=NULL, dq=NULL, gk=NULL, gv=NULL)
    assert backward(B=0, **none, decay=NULL, state0=NULL, dstate=NULL, dstate0=NULL, ddecay=NULL, ws=NULL) == 0
    assert backward(T=0, **none, decay=NULL, state0=NULL, dstate=NULL, dstate0=NULL, ddecay=NULL, ws=NULL) == 0
    # the states' gradients remain without tokens: these two enqueue work, and fail for lack of a device
    assert backward(T=0, **none, ddecay=NULL) == HIP
    assert backward(B=0, **none, decay=NULL, dstate0=NULL) == HIP
    assert backward() == HIP
    assert backward(state0=NULL, dstate=NULL, dstate0=NULL, ddecay=NULL, lengths=NULL) == HIP


def norm(rows=8, G=2, C=24, x=P(0), dt=F32, w=P(16 * MB), b=P(32 * MB), y=P(48 * MB), mean=P(64 * MB),
         rstd=P(80 * MB), eps=1e-5):
    return ln._lib().gdn_layer_norm(rows, G, C, x, dt, w, b, y, mean, rstd, eps, None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(rows=-1), INVALID, "rows"),
    (dict(rows=7), INVALID, "multiple of G"),
    (dict(G=0), INVALID, "G and C"),
    (dict(C=0), INVALID, "G and C"),
    (dict(G=1 << 20, C=1 << 20, rows=1 << 20), INVALID, "G * C"),
    (dict(rows=1 << 60), INVALID, "overflows"),
    (dict(dt=5), INVALID, "dtype"),
    (dict(eps=-1.0), INVALID, "eps"),
    (dict(eps=float("nan")), INVALID, "eps"),
    (dict(mean=NULL), INVALID, "together"),
    (dict(x=NULL), INVALID, "x is NULL"),
    (dict(y=NULL), INVALID, "y is NULL"),
    (dict(w=P(16 * MB + 4)), INVALID, "weight is not 16-byte aligned"),
    (dict(y=P(16)), INVALID, "y overlaps x"),
    (dict(y=P(16 * MB)), INVALID, "y overlaps weight"),
    (dict(mean=P(48 * MB)), INVALID, "y overlaps mean"),
    (dict(mean=P(0)), INVALID, "mean overlaps x"),
    (dict(mean=P(80 * MB)), INVALID, "mean overlaps rstd"),
])
@fake_ptrs
def test_layer_norm_rejects(kw, status, msg):
    assert norm(**kw) == status
    assert msg in last_error()


@fake_ptrs
def test_layer_norm_empty_work_and_calls_without_a_device():
    assert norm(rows=0, x=NULL, y=NULL, w=NULL, b=NULL, mean=NULL, rstd=NULL) == 0
    assert norm() == HIP
    assert norm(y=P(0)) == HIP   # in place
    assert norm(w=NULL, b=NULL, mean=NULL, rstd=NULL) == HIP


def norm_backward(rows=8, G=2, C=24, dy=P(0), x=P(16 * MB), dt=F32, w=P(32 * MB), mean=P(48 * MB), rstd=P(64 * MB),
                  dx=P(80 * MB), dw=P(96 * MB), db=P(112 * MB), ws=P(1 << 40), wsb=1 << 40):
    return ln._lib().gdn_layer_norm_backward(rows, G, C, dy, x, dt, w, mean, rstd, dx, dw, db, ws, wsb, None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(rows=-2), INVALID, "rows"),
    (dict(rows=9), INVALID, "multiple of G"),
    (dict(dt=-1), INVALID, "dtype"),
    (dict(mean=NULL), INVALID, "mean is NULL"),
    (dict(dx=NULL), INVALID, "dx is NULL"),
    (dict(dw=P(96 * MB + 4)), INVALID, "dweight is not 16-byte aligned"),
    (dict(dx=P(16 * MB)), INVALID, "dx overlaps x"),
    (dict(dx=P(16)), INVALID, "dx overlaps dy"),
    (dict(dw=P(112 * MB)), INVALID, "dweight overlaps dbias"),
    (dict(db=P(32 * MB)), INVALID, "dbias overlaps weight"),
    (dict(ws=NULL), INVALID, "workspace is NULL"),
    (dict(wsb=16), INVALID, "needed"),
    (dict(ws=P(80 * MB)), INVALID, "dx overlaps workspace"),
])
@fake_ptrs
def test_layer_norm_backward_rejects(kw, status, msg):
    assert norm_backward(**kw) == status
    assert msg in last_error()


@fake_ptrs
def test_layer_norm_backward_empty_work_and_calls_without_a_device():
    assert norm_backward(rows=0, dy=NULL, x=NULL, mean=NULL, rstd=NULL, dx=NULL, dw=NULL, db=NULL, ws=NULL) == 0
    assert norm_backward(rows=0, dy=NULL, x=NULL, mean=NULL, rstd=NULL, dx=NULL) == HIP   # zeros dweight, dbias
    assert norm_backward() == HIP
    assert norm_backward(dx=P(0)) == HIP   # over dy
    assert norm_backward(dw=NULL, db=NULL, ws=NULL, wsb=0) == HIP


@pytest.mark.parametrize("fn,args", [
    (lambda: gdn.linear_attn_prefill_workspace_size, (1, 8, 4, 48, 48)),
    (lambda: gdn.linear_attn_backward_workspace_size, (1, 8, 4, 3, 16, 16)),
    (lambda: gdn.layer_norm_backward_workspace_size, (7, 2, 16)),
])
def test_workspace_sizes_reject(fn, args):
    with pytest.raises(gdn.GDNError):
        fn()(*args)


def test_workspace_sizes():
    assert gdn.linear_attn_prefill_workspace_size(0, 8, 4, 16, 16) == 0
    # two fp32 gradients of every head where heads share q and k
    assert gdn.linear_attn_backward_workspace_size(2, 8, 4, 2, 16, 16) >= 2 * 2 * 8 * 4 * 16 * 4
    assert gdn.layer_norm_backward_workspace_size(8, 2, 24) >= 2 * 2 * 24 * 4
    for fn in ("gdn_linear_attn_prefill_workspace_size", "gdn_layer_norm_backward_workspace_size"):
        args = (1, 8, 4, 16, 16) if "attn" in fn else (8, 2, 16)
        assert getattr(ln._lib(), fn)(*args, None) == INVALID and "bytes is NULL" in last_error()


def test_binding_rejects_cpu_tensors_and_bad_shapes():
    q = torch.zeros(1, 2, 2, 16)
    with pytest.raises(ValueError, match="HIP device"):
        gdn.linear_attn_decode_step(q, q, q, torch.zeros(2), torch.zeros(1, 2, 16, 16))
    with pytest.raises(ValueError, match="q must be"):
        gdn.linear_attn_prefill(q[0], q, q, torch.zeros(2), torch.zeros(1, 2, 16, 16))
    with pytest.raises(ValueError, match="v must be"):
        gdn.linear_attn_backward(q, q, q[0], torch.zeros(2), q)
    with pytest.raises(ValueError, match="HIP device"):
        gdn.layer_norm(torch.zeros(4, 8))
    with pytest.raises(ValueError, match="x must be"):
        gdn.layer_norm_backward(3.0, 3.0, None, None)


def test_workspace_of_large_affines():
    # no more slabs than rows of a group, and slabs * G * C within one launch
    assert gdn.layer_norm_backward_workspace_size(0, 4, 64) == 0
    assert gdn.layer_norm_backward_workspace_size(12, 4, 64) == 2 * 3 * 4 * 64 * 4
    assert gdn.layer_norm_backward_workspace_size(256 * 2048, 2048, 8192) == 2 * 128 * (1 << 24) * 4
    assert gdn.layer_norm_backward_workspace_size(1 << 20, 1, (1 << 31) - 1) == 2 * ((1 << 31) - 1) * 4
