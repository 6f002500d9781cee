"""Tensors of more than 2^31 values: the rotation, the norm and the gated recurrence against the same calls on their last
rows and channels."""
import pytest
import torch

import gated_deltanet_recurrent_02_amd as gdn

pytestmark = pytest.mark.gpu


def big(*shape, seed):
    """bf16 values on the GPU, drawn in slices so that no fp32 copy of the whole exists."""
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(seed)
    for part in out.view(-1).split(1 << 28):
        part.normal_(generator=g)
    return out


def test_rotation_and_norm_past_2_31_values():
    T, H, Hk, D = 271000, 62, 2, 128
    assert T * H * D > 2 ** 31
    q, k = big(1, T, H, D, seed=1), big(1, T, Hk, D, seed=2)
    freqs = gdn.rope_frequencies(D)[0].cuda()
    w = torch.rand(D, device="cuda")
    n = 50
    last = torch.arange(T - n, T, dtype=torch.int32, device="cuda")[None]
    y, z = gdn.rope(q, k, freqs)
    a, b = gdn.rope(q[:, -n:], k[:, -n:], freqs, positions=last)
    assert torch.equal(y[:, -n:], a) and torch.equal(z[:, -n:], b)
    gdn.qk_norm_rope(q, k, freqs, q_weight=w, q_out=y, k_out=z)
    a, b = gdn.qk_norm_rope(q[:, -n:], k[:, -n:], freqs, positions=last, q_weight=w)
    assert torch.equal(y[:, -n:], a) and torch.equal(z[:, -n:], b)
    # gradients over themselves; only the last rows' are not zero, so that the weights' sums are theirs
    y[:, :-n].zero_()
    d = y[:, -n:].clone()
    gq, _, dw, _ = gdn.qk_norm_rope_backward(y, torch.zeros_like(z), q, k, freqs, q_weight=w, q_out=y)
    a, _, dw2, _ = gdn.qk_norm_rope_backward(d, None, q[:, -n:], None, freqs, positions=last, q_weight=w)
    assert gq is y and torch.equal(y[:, -n:], a) and not y[:, :-n].any()
    # the same 3100 terms in another order: at most 3100 roundings of 2^-24 of their sizes' sum, with ten times that of room
    torch.testing.assert_close(dw, dw2, rtol=1e-3, atol=1e-3 * dw2.abs().max().item())


@pytest.mark.parametrize("B,T,C", [(1, 33000, 66000), (3, 33000, 22001)])
def test_recurrence_past_2_31_values(B, T, C):
    assert B * T * C > 2 ** 31
    x, a = big(B, T, C, seed=3), big(B, T, C, seed=4)
    rate = torch.rand(C, device="cuda") + 0.1
    s = torch.randn(B, C, device="cuda")
    n = 130
    cut = (slice(B - 1, B), slice(None), slice(C - n, C))
    part = s[cut[0], cut[2]].clone()
    o = gdn.gated_scan_prefill(x, a, None, s, rate=rate)
    ref = gdn.gated_scan_prefill(x[cut], a[cut], None, part, rate=rate[-n:].clone())
    # two correct results differ by two half steps of bf16 at most, and by their bars of fp32
    torch.testing.assert_close(o[cut].float(), ref.float(), rtol=2.0 ** -7, atol=1e-5)
    torch.testing.assert_close(s[cut[0], cut[2]], part, rtol=1e-5, atol=1e-6)
    dx, da, _, _, drate = gdn.gated_scan_backward(x, a, None, o, rate=rate, rate_grad=True)
    px, pa, _, _, prate = gdn.gated_scan_backward(x[cut], a[cut], None, o[cut], rate=rate[-n:].clone(), rate_grad=True)
    torch.testing.assert_close(dx[cut].float(), px.float(), rtol=2.0 ** -7, atol=1e-5)
    torch.testing.assert_close(da[cut].float(), pa.float(), rtol=2.0 ** -7, atol=1e-5)
    if B == 1:
        torch.testing.assert_close(drate[-n:], prate, rtol=1e-4, atol=1e-4 * prate.abs().max().item())
