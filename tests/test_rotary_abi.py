"""The C ABI of include/gdn_rotary.h on the CPU: exports, refusals of invalid arguments before any HIP
call, strided views told apart, empty work, workspace sizes, the binding's own checks, and the
frequencies against their formulas."""
import ctypes
import math
import os
import re

import pytest
import torch

import gated_deltanet_recurrent_02_amd as gdn
from gated_deltanet_recurrent_02_amd import _binding as bd
from gated_deltanet_recurrent_02_amd import _rotary as ro

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdn_rotary.h")
INVALID, UNSUPPORTED, HIP = bd.GDN_ERR_INVALID_ARGUMENT, bd.GDN_ERR_UNSUPPORTED, bd.GDN_ERR_HIP
F32, BF16 = bd.GDN_F32, bd.GDN_BF16
BASE = 0x7F0000000000  # a fake, 256-byte aligned device address
MB = 1 << 20
NULL = ctypes.c_void_p(0)

# Fake device pointers are only ever passed where no GPU is visible.
fake_ptrs = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="passes fake device pointers")


def P(off=0):
    return ctypes.c_void_p(BASE + off)


def S(*strides):
    return ro._pack3(*strides)


def last_error():
    return gdn.lib().gdn_last_error().decode()


def test_header_declares_the_binding_exports():
    with open(HEADER) as f:
        text = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(gdn_[a-z0-9_]+)\s*\(", text)))
    assert declared == sorted(gdn.ROTARY_EXPORTS)
    L = ctypes.CDLL(bd.LIBRARY)
    for name in declared:
        assert hasattr(L, name), name


SIZES = dict(B=2, T=4, Hq=4, Hk=2, D=16, R=16, dt=F32)
REST = dict(pos=P(64 * MB), freqs=P(65 * MB), amp=1.0, inter=0, lengths=P(66 * MB))


def call(kind="gdn_rope", B=2, T=4, Hq=4, Hk=2, D=16, R=16, dt=F32, q=P(0), qs=None, k=P(16 * MB), ks=None, dq=P(200 * MB),
         dqs=None, dk=P(210 * MB), dks=None, wq=P(220 * MB), wk=P(221 * MB), per_head=0, eps=1e-6, pos=P(64 * MB),
         freqs=P(65 * MB), amp=1.0, inter=0, lengths=P(66 * MB), qo=P(80 * MB), qos=None, ko=P(96 * MB), kos=None,
         gq=P(230 * MB), gk=P(231 * MB), ws=P(1 << 40), wsb=1 << 40):
    L = ro._lib()
    sizes, turn, out = (B, T, Hq, Hk, D, R, dt), (pos, freqs, amp, inter, lengths), (qo, qos, ko, kos)
    if kind in ("gdn_rope", "gdn_rope_backward"):
        return getattr(L, kind)(*sizes, q, qs, k, ks, *turn, *out, None)
    if kind == "gdn_qk_norm_rope":
        return L.gdn_qk_norm_rope(*sizes, q, qs, k, ks, wq, wk, per_head, eps, *turn, *out, None)
    return L.gdn_qk_norm_rope_backward(*sizes, dq, dqs, dk, dks, q, qs, k, ks, wq, wk, per_head, eps, *turn, *out, gq, gk,
                                       ws, wsb, None)


KINDS = ["gdn_rope", "gdn_rope_backward", "gdn_qk_norm_rope", "gdn_qk_norm_rope_backward"]
NORMS = KINDS[2:]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("kw,status,msg", [
    (dict(B=-1), INVALID, "B and T"),
    (dict(T=-1), INVALID, "B and T"),
    (dict(Hq=0), INVALID, "Hq"),
    (dict(Hk=-1), INVALID, "Hk"),
    (dict(D=0), INVALID, "D must be"),
    (dict(D=513), UNSUPPORTED, "D must be"),
    (dict(Hq=1 << 14), UNSUPPORTED, "Hq + Hk"),
    (dict(Hq=(1 << 31) - 1, Hk=(1 << 31) - 1), UNSUPPORTED, "Hq + Hk"),
    (dict(B=1 << 31), UNSUPPORTED, "B * T"),
    (dict(B=1 << 62), UNSUPPORTED, "B * T"),
    (dict(B=2, T=1 << 30), UNSUPPORTED, "B * T"),
    (dict(R=15), INVALID, "R must be"),
    (dict(R=18), INVALID, "R must be"),
    (dict(R=-2), INVALID, "R must be"),
    (dict(dt=3), INVALID, "dtype"),
    (dict(dt=-1), INVALID, "dtype"),
    (dict(amp=float("nan")), INVALID, "amplitude"),
    (dict(amp=float("inf")), INVALID, "amplitude"),
    (dict(freqs=NULL), INVALID, "freqs is NULL"),
    (dict(freqs=P(65 * MB + 8)), INVALID, "freqs is not 16-byte aligned"),
    (dict(pos=P(64 * MB + 4)), INVALID, "positions is not 16-byte aligned"),
    (dict(lengths=P(66 * MB + 4)), INVALID, "lengths is not 16-byte aligned"),
    (dict(qo=NULL), INVALID, "q_out is NULL"),
    (dict(ko=P(96 * MB + 2)), INVALID, "k_out is not aligned"),
    (dict(qos=S(64, -16, 16)), INVALID, "negative stride"),
    (dict(qos=S(1 << 62, 64, 16)), INVALID, "overflows"),
    (dict(qos=S(1 << 59, 64, 16)), INVALID, "overflows"),
    (dict(qos=S(256, 64, 0)), INVALID, "q_out overlap each other"),
    (dict(qos=S(256, 64, 8)), INVALID, "q_out overlap each other"),
    (dict(qos=S(64, 64, 16)), INVALID, "q_out overlap each other"),
    (dict(qos=S(192, 64, 16)), INVALID, "q_out overlap each other"),
    (dict(qo=P(96 * MB)), INVALID, "q_out overlaps k_out"),
    (dict(qo=P(64 * MB)), INVALID, "q_out overlaps positions"),
    (dict(ko=P(65 * MB)), INVALID, "k_out overlaps freqs"),
    (dict(ko=P(66 * MB)), INVALID, "k_out overlaps lengths"),
])
@fake_ptrs
def test_rejects(kind, kw, status, msg):
    assert call(kind, **kw) == status
    assert msg in last_error()


@pytest.mark.parametrize("kind", KINDS[:3])
@pytest.mark.parametrize("kw,msg", [
    (dict(q=NULL), " is NULL"),
    (dict(q=P(2)), " is not aligned"),
    (dict(qs=S(64, 16, -1)), "negative stride"),
    (dict(qo=P(16 * MB)), "q_out overlaps"),          # over k
    (dict(qo=P(64)), "q_out overlaps"),               # over q, but not in place
    (dict(qo=P(0), qos=S(1024, 64, 16)), "q_out overlaps"),
    (dict(q=P(0), k=P(0), qo=P(0)), "q_out overlaps"),  # in place while k is the same tensor
])
@fake_ptrs
def test_forward_rejects(kind, kw, msg):
    assert call(kind, **kw) == INVALID
    assert msg in last_error()


@pytest.mark.parametrize("kind", NORMS)
@pytest.mark.parametrize("kw,msg", [
    (dict(eps=-1e-6), "eps"),
    (dict(eps=float("nan")), "eps"),
    (dict(wq=P(220 * MB + 4)), "q_weight is not 16-byte aligned"),
    (dict(qo=P(220 * MB)), "q_out overlaps q_weight"),
    (dict(ko=P(221 * MB)), "k_out overlaps k_weight"),
])
@fake_ptrs
def test_norm_rejects(kind, kw, msg):
    assert call(kind, **kw) == INVALID
    assert msg in last_error()


@pytest.mark.parametrize("kw,msg", [
    (dict(dq=NULL), "dq is NULL"),
    (dict(q=NULL), "q is NULL"),
    (dict(gq=P(230 * MB + 8)), "dq_weight is not 16-byte aligned"),
    (dict(gq=P(231 * MB)), "dq_weight overlaps dk_weight"),
    (dict(gk=P(220 * MB)), "dk_weight overlaps q_weight"),
    (dict(gq=P(0)), "dq_weight overlaps q"),
    (dict(qo=P(0)), "q_out overlaps q"),               # in place is over dq
    (dict(ko=P(210 * MB + 64)), "k_out overlaps dk"),
    (dict(ws=NULL), "workspace is NULL"),
    (dict(wsb=64), "needed"),
    (dict(ws=P(80 * MB)), "q_out overlaps workspace"),
    (dict(ws=P(0)), "workspace overlaps q"),
])
@fake_ptrs
def test_norm_backward_rejects(kw, msg):
    assert call("gdn_qk_norm_rope_backward", **kw) == INVALID
    assert msg in last_error()


@pytest.mark.parametrize("kind", KINDS)
@fake_ptrs
def test_valid_calls_without_a_device(kind):
    """Accepted, and then there is no device: what the documentation allows."""
    tok = (4 + 2 + 2) * 16     # q, k and v parts of a packed projection
    packed = dict(q=P(0), qs=S(4 * tok, tok, 16), k=P(64 * 4), ks=S(4 * tok, tok, 16))
    into = dict(qo=P(300 * MB), qos=S(4 * tok, tok, 16), ko=P(300 * MB + 64 * 4), kos=S(4 * tok, tok, 16))
    for kw in (dict(), dict(pos=NULL, lengths=NULL), dict(R=0, freqs=NULL), dict(Hk=0, k=NULL, ko=NULL, wk=NULL),
               dict(inter=1, D=33, R=32), packed, into, dict(packed, **into), dict(wq=NULL, wk=NULL), dict(per_head=1),
               dict(q=P(4), qs=S(1024, 64, 16)),                                   # aligned to its element only
               dict(qo=P(80 * MB), qos=S(16, 32, 16 * 2 * 4)),                     # another order of dimensions
               dict(qs=S(0, 0, 0)),                                                # a broadcast input
               dict(qo=P(80 * MB), qos=S(256 * 2, 64 * 2, 32), ko=P(80 * MB + 64), kos=S(256 * 2, 64 * 2, 32), Hk=4)):
        assert call(kind, **kw) == HIP, (kw, last_error())
    place = dict(q=P(0), k=P(16 * MB)) if kind != KINDS[3] else dict(dq=P(0), dk=P(16 * MB), q=P(300 * MB), k=P(310 * MB))
    assert call(kind, **place, qo=P(0), ko=P(16 * MB)) == HIP                      # in place
    # in place in a packed tensor
    if kind != KINDS[3]:
        assert call(kind, **packed, qo=P(0), qos=packed["qs"], ko=P(64 * 4), kos=packed["ks"]) == HIP, last_error()
        shifted = dict(packed, k=P(64 * 4 - 4))
        assert call(kind, **shifted, qo=P(0), qos=packed["qs"]) == INVALID and "q_out overlaps" in last_error()


@pytest.mark.parametrize("kind", KINDS)
@fake_ptrs
def test_empty_work(kind):
    none = dict(q=NULL, k=NULL, dq=NULL, dk=NULL, qo=NULL, ko=NULL, pos=NULL, freqs=NULL, lengths=NULL, wq=NULL, wk=NULL, ws=NULL, wsb=0)
    for B, T in ((0, 3), (2, 0), (0, 0)):
        assert call(kind, B=B, T=T, **none, gq=NULL, gk=NULL) == 0 and last_error() == ""
    if kind == KINDS[3]:
        assert call(kind, B=0, **none) == HIP     # zeros the weights' gradients
        assert call(kind, T=0, **none, gk=NULL) == HIP


def test_workspace_sizes():
    size = gdn.qk_norm_rope_backward_workspace_size
    assert size(0, 8, 4, 2, 16) == 0 and size(2, 0, 4, 2, 16) == 0
    assert size(1, 3, 4, 2, 16) == (3 + 1) * 6 * 16 * 4
    assert size(1 << 30, 1, 16000, 384, 512) == 257 * 16384 * 512 * 4
    assert size(4, 4096, 48, 16, 128) == 257 * 64 * 128 * 4
    assert size(4, 4096, 1, 0, 128) == 1025 * 128 * 4
    with pytest.raises(gdn.GDNError):
        size(1, 8, 0, 2, 16)
    assert ro._lib().gdn_qk_norm_rope_backward_workspace_size(1, 8, 4, 2, 16, None) == INVALID
    assert "bytes is NULL" in last_error()


def test_binding_rejects_cpu_tensors_and_bad_shapes():
    q, f = torch.zeros(1, 2, 2, 16), torch.zeros(8, dtype=torch.float64)
    with pytest.raises(ValueError, match="HIP device"):
        gdn.rope(q, q, f)
    with pytest.raises(ValueError, match="q must be"):
        gdn.rope(q[0], q, f)
    with pytest.raises(ValueError, match="dk must be"):
        gdn.rope_backward(q, q[0], f)
    with pytest.raises(ValueError, match="freqs"):
        gdn.rope(q, q, None)
    with pytest.raises(ValueError, match="HIP device"):
        gdn.qk_norm_rope(q, None)
    with pytest.raises(ValueError, match="together"):
        gdn.qk_norm_rope_backward(q, None, q, q)


def test_frequencies():
    f, amp = gdn.rope_frequencies(8, base=100.0)
    assert f.dtype is torch.float64 and amp == 1.0
    assert f.tolist() == pytest.approx([1.0, 100 ** -0.25, 100 ** -0.5, 100 ** -0.75], rel=1e-15)
    lin, _ = gdn.rope_frequencies(8, base=100.0, scaling="linear", factor=4.0)
    assert torch.allclose(lin * 4, f, rtol=1e-15, atol=0)
    ntk, _ = gdn.rope_frequencies(8, base=100.0, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0 and float(f[-1] / ntk[-1]) == pytest.approx(4.0, rel=1e-12)
    yarn, amp = gdn.rope_frequencies(64, scaling="yarn", factor=8.0, original_length=4096)
    f, _ = gdn.rope_frequencies(64)
    assert amp == pytest.approx(0.1 * math.log(8.0) + 1)
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(yarn[turns >= 32], f[turns >= 32])
    assert torch.allclose(yarn[turns <= 1], f[turns <= 1] / 8, rtol=1e-15, atol=0)
    mid = (turns > 1) & (turns < 32)
    keep = (turns[mid] - 1) / 31
    assert mid.any() and torch.allclose(yarn[mid], f[mid] * (keep + (1 - keep) / 8), rtol=1e-14, atol=0)


@pytest.mark.parametrize("args,msg", [
    (dict(dim=7), "dim"), (dict(dim=0), "dim"), (dict(dim=8, base=-1.0), "base"), (dict(dim=8, factor=0.5), "factor"),
    (dict(dim=8, scaling="cubic"), "scaling"), (dict(dim=2, scaling="ntk", factor=2.0), "ntk"),
    (dict(dim=8, scaling="yarn", factor=2.0), "original_length"),
    (dict(dim=8, scaling="yarn", factor=2.0, original_length=64, beta_fast=1.0), "beta_fast")])
def test_frequencies_reject(args, msg):
    with pytest.raises(ValueError, match=msg):
        gdn.rope_frequencies(**args)
