"""The arithmetic of the attention on the tensor cores, modelled on the CPU in 64 bits: every f32 as
two f16 with a power-of-two scale, three of the four partial products.  It is as good as plain f32
by the comparison that the GPU tests use, and that comparison rejects every form that drops one of
the low halves."""
import pytest
import torch

import attention_forms as forms

TILE = 64


def two_f16(x, top):
    """hi, lo (64-bit, unscaled) of x scaled so that top, broadcast, is in [2^14, 2^15)."""
    e = 14 - torch.floor(torch.log2(top.double().clamp_min(1e-300)))
    f = torch.exp2(e)
    y = x.double() * f
    hi = y.half().double()
    lo = (y - hi).half().double()
    return hi / f, lo / f


def product(a, b, drop):
    """a @ b of (hi, lo) pairs without lo lo, and without what `drop` names."""
    (ah, al), (bh, bl) = a, b
    out = ah @ bh
    if "a" not in drop:
        out = out + al @ bh
    if "b" not in drop:
        out = out + ah @ bl
    return out


def model(q, k, v, seen, scale, cap, drop=""):
    """One head.  drop: letters of q, k, p, v whose low half is left out."""
    s = product(two_f16(q, q.abs().amax(-1, keepdim=True)),
                tuple(t.T for t in two_f16(k, k.abs().amax(-1, keepdim=True))),
                {"q": "a", "k": "b"}.get(drop, "ab" if drop == "qk" else "")) * scale
    if cap:
        s = cap * torch.tanh(s / cap)
    s = s.masked_fill(~seen, -float("inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True)).float()
    out = torch.zeros(q.shape, dtype=torch.float64)
    for t in range(0, k.shape[0], TILE):
        vt = v[t:t + TILE]
        out += product(two_f16(p[:, t:t + TILE], torch.ones(1)), two_f16(vt, vt.abs().amax()),
                       {"p": "a", "v": "b"}.get(drop, "ab" if drop == "pv" else ""))
    return out / p.double().sum(-1, keepdim=True)


CASES = [(777, 777, 256, 0.0), (300, 300, 256, 50.0), (300, 900, 128, 0.0), (400, 400, 64, 1.5),
         (400, 400, 32, 0.0), (130, 4000, 256, 0.0)]


def inputs(nq, nk, hd):
    g = torch.Generator().manual_seed(84000 + nq + hd)
    return [torch.randn(n, hd, generator=g) for n in (nq, nk, nk)]


@pytest.mark.parametrize("nq,nk,hd,cap", CASES)
def test_the_split_is_as_good_as_f32(nq, nk, hd, cap):
    q, k, v = inputs(nq, nk, hd)
    seen, s = forms.causal(nq, nk, "cpu"), hd ** -0.5
    ref = forms.attend(q, k, v, seen, s, cap)
    plain = forms.attend(q, k, v, seen, s, cap, torch.float32)
    forms.assert_as_good_as_f32(model(q, k, v, seen, s, cap), plain, ref)


@pytest.mark.parametrize("drop", ["q", "k", "p", "v", "qk", "pv"])
@pytest.mark.parametrize("nq,nk,hd,cap", CASES)
def test_a_low_half_left_out_is_seen(nq, nk, hd, cap, drop):
    q, k, v = inputs(nq, nk, hd)
    seen, s = forms.causal(nq, nk, "cpu"), hd ** -0.5
    ref = forms.attend(q, k, v, seen, s, cap)
    plain = forms.attend(q, k, v, seen, s, cap, torch.float32)
    with pytest.raises(AssertionError):
        forms.assert_as_good_as_f32(model(q, k, v, seen, s, cap, drop), plain, ref)
