"""The checks of strided tensors behind the C ABI (gdn_strided.h) against brute force: a call whose output shares a byte
with another argument, or with itself, is refused, whatever the strides; interleaved views that share nothing are taken."""
import ctypes
import random

import pytest
import torch

import gated_deltanet_recurrent_02_amd as gdn
from gated_deltanet_recurrent_02_amd import _binding as bd
from gated_deltanet_recurrent_02_amd import _rotary as ro
from gated_deltanet_recurrent_02_amd import _scan as sc

BASE = 0x7F0000000000
MB = 1 << 20
ACCEPTED, REFUSED = bd.GDN_ERR_HIP, bd.GDN_ERR_INVALID_ARGUMENT   # accepted: then there is no device

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="passes fake device pointers")


def P(off):
    return ctypes.c_void_p(BASE + off)


def elements(start, sizes, strides, row):
    """Element numbers of a strided tensor, with repetitions."""
    at = [start]
    for n, s in zip(sizes, strides):
        at = [p + i * s for p in at for i in range(n)]
    return [p + c for p in at for c in range(row)]


def test_rows_against_brute_force():
    rng = random.Random(1)
    counts = {True: 0, False: 0}
    for _ in range(4000):
        B, T, C = rng.randint(1, 3), rng.randint(1, 4), rng.randint(1, 4)

        def strides():
            st = rng.choice([C, 2 * C, 3 * C, rng.randint(0, 12)])
            return rng.choice([T * st, (T + 1) * st, 4 * C, rng.randint(0, 50)]), st
        xs, os = strides(), rng.choice([strides(), None])
        if os is None:
            os = xs
        off = rng.randint(0, 40)
        x = elements(100, (B, T), xs, C)
        o = elements(100 + off, (B, T), os, C)
        clash = len(set(o)) < len(o) or bool(set(x) & set(o))
        status = sc._lib().gdn_gated_scan_decode_step(B, T, C, P(400), sc._pack2(*xs), P(MB), None, None, None, 0, None, None,
                                                      P(2 * MB), 0, P(4 * (100 + off)), sc._pack2(*os), None)
        if clash:
            assert status == REFUSED, (B, T, C, xs, os, off)
        counts[status == ACCEPTED] += 1
    assert counts[True] > 300 and counts[False] > 300


def test_heads_against_brute_force():
    rng = random.Random(2)
    accepted = 0
    for _ in range(4000):
        B, T, Hq, Hk, D = (rng.randint(1, 3) for _ in range(5))
        R = D // 2 * 2
        unit = (Hq + Hk + rng.randint(0, 2)) * D

        def view(H):
            kind = rng.randint(0, 3)
            if kind == 0:       # part of a packed projection
                return (T * unit, unit, D)
            if kind == 1:       # heads before tokens
                return (unit * T, D, T * D)
            if kind == 2:       # heads interleaved with something else
                return (T * H * 2 * D, H * 2 * D, 2 * D)
            return tuple(rng.randint(0, 30) for _ in range(3))
        qs, ks = view(Hq), view(Hk)
        off = rng.choice([Hq * D, D, 0, rng.randint(0, 60)])
        q, k = elements(0, (B, T, Hq), qs, D), elements(off, (B, T, Hk), ks, D)
        clash = len(set(q)) < len(q) or len(set(k)) < len(k) or bool(set(q) & set(k))
        f, out = P(8 * MB), (P(0), ro._pack3(*qs), P(4 * off), ro._pack3(*ks))
        status = ro._lib().gdn_rope(B, T, Hq, Hk, D, R, 0, *out, None, f, 1.0, 0, None, *out, None)     # in place
        if clash:
            assert status == REFUSED, (B, T, Hq, Hk, D, qs, ks, off)
        accepted += status == ACCEPTED
    assert accepted > 300


def test_views_of_one_tensor_are_taken():
    """Parts of a packed tensor, heads between heads, and a tensor between another's sequences."""
    B, T, H, D = 3, 5, 4, 8
    f = P(8 * MB)

    def rope(q, qs, k, ks):
        out = (P(4 * q), ro._pack3(*qs), P(4 * k), ro._pack3(*ks))
        return ro._lib().gdn_rope(B, T, H, H, D, D, 0, *out, None, f, 1.0, 0, None, *out, None)

    packed = (T * 3 * H * D, 3 * H * D, D)
    assert rope(0, packed, H * D, packed) == ACCEPTED
    assert rope(0, packed, H * D - 1, packed) == REFUSED
    pairs = (T * 2 * H * D, 2 * H * D, 2 * D)
    assert rope(0, pairs, D, pairs) == ACCEPTED
    assert rope(D, pairs, 0, pairs) == ACCEPTED
    first = (2 * H * T * D, D, T * D)          # [B][2 H][T][D], the first and the second H heads
    assert rope(0, first, H * T * D, first) == ACCEPTED
    assert rope(H * T * D, first, 0, first) == ACCEPTED
    assert rope(0, first, H * T * D - D, first) == REFUSED
    assert gdn.lib().gdn_last_error().decode()
