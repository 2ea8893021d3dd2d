"""How far prompt_attention and prefix_attention on the tensor cores are from 64 bits: on ordinary
inputs no further than a few times plain f32 (test_split_model.py shows that this sees any low half
that is left out), and at the border of the range that qws.h states for channels of very different
size."""
import pytest
import torch

import attention_forms as forms
from quantized_weight_streaming_q4k_gb300 import build, ops

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    torch.cuda.set_device(0)
    assert not torch.backends.cuda.matmul.allow_tf32
    yield
    assert ops.device_error() == 0


def normal(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(85000 + seed)
    return torch.randn(shape, device="cuda", generator=g)


# ------------------------------------------------------------------ ordinary inputs
@pytest.mark.parametrize("cap", [0.0, 50.0, 1.5])
@pytest.mark.parametrize("nq,nkv,hd", [(8, 4, 256), (16, 4, 128), (6, 2, 64), (2, 1, 32)])
def test_prompt(nq, nkv, hd, cap):
    cu, s = [0, 900, 1200], hd ** -0.5
    q, k, v = normal(1, 1200, nq, hd), normal(2, 1200, nkv, hd), normal(3, 1200, nkv, hd)
    got = ops.prompt_attention(q, k, v, cu, s, cap)
    ref = forms.prompt_forms(q, k, v, cu, cu, s, cap, torch.float64)
    forms.assert_as_good_as_f32(got, forms.prompt_forms(q, k, v, cu, cu, s, cap, torch.float32), ref)


@pytest.mark.parametrize("nq,nkv,hd", [(8, 4, 256), (4, 1, 64)])
def test_prompt_continued_in_pieces(nq, nkv, hd):
    cu, ck, s = [0, 130], [0, 4000], hd ** -0.5
    q, k, v = normal(4, 130, nq, hd), normal(5, 4000, nkv, hd), normal(6, 4000, nkv, hd)
    got = ops.prompt_attention(q, k, v, cu, s, cu_seqlens_k=ck)
    ref = forms.prompt_forms(q, k, v, cu, ck, s, 0.0, torch.float64)
    forms.assert_as_good_as_f32(got, forms.prompt_forms(q, k, v, cu, ck, s, 0.0, torch.float32), ref)


@pytest.mark.parametrize("cap", [0.0, 50.0])
@pytest.mark.parametrize("nq,nkv,hd", [(8, 4, 256), (16, 4, 128), (6, 2, 64), (2, 1, 32)])
def test_prefix(nq, nkv, hd, cap):
    B, P = 9, 3000
    n_ctx = [0, 40, 7, 1, 33, 64, 2, 19, 5]
    q, kp, vp = normal(7, B, nq, hd), normal(8, nkv, P, hd), normal(9, nkv, P, hd)
    kc, vc = normal(10, B, nkv, 64, hd), normal(11, B, nkv, 64, hd)
    args = (q, kp, vp, P, kc, vc, n_ctx, hd ** -0.5, cap)
    ref = forms.prefix_forms(*args, torch.float64)
    forms.assert_as_good_as_f32(ops.prefix_attention(*args),
                                forms.prefix_forms(*args, torch.float32), ref)


@pytest.mark.parametrize("nq,nkv,hd", [(8, 4, 256), (8, 2, 64), (8, 4, 128)])
def test_prompt_rows_equal_kv_attention(nq, nkv, hd):
    n, s = 1300, hd ** -0.5
    q, kc, vc = normal(12, n, nq, hd), normal(13, nkv, n, hd), normal(14, nkv, n, hd)
    got = ops.prompt_attention(q, kc.transpose(0, 1), vc.transpose(0, 1), [0, n], s)
    for i in (0, 1, 63, 64, 127, 128, 500, n - 1):
        one = ops.kv_attention(q[i].contiguous(), kc, vc, nq, nkv, hd, n, i + 1, s)
        # both within 1e-6 of values up to 5 (their own errors are some 1e-6 at most)
        assert torch.all((got[i] - one).abs() <= 1e-5)


# ------------------------------------------------------------------ channels of very different size
def head_bound(q, k, v, seen, s, k_range, v_error):
    """(reference, largest error) of a head from what qws.h states: a score is within
    (hd + 32) u max_t sum |s q k| + |s| sum_i (dq_i |k_ti| + |q_i| dk_ti) of its own, where dq is
    2^-39 of the row's largest and dk k_range of it (the rest of dq and dk, 2^-22 of the value
    itself, is in the first term); weights e^(+-2 ds); a value within v_error or 2^-22 of itself;
    sums 1e-5 of sum p |v| as in test_gpu_prompt."""
    ref = forms.attend(q, k, v, seen, s)
    Q, K, V = q.double().abs(), k.double().abs(), v.double()
    size = abs(s) * (Q @ K.T)
    ds = (q.shape[-1] + 32) * U * size.masked_fill(~seen, 0.0).amax(-1, keepdim=True)
    ds = ds + abs(s) * (2.0 ** -39 * Q.amax(-1, keepdim=True) * K.sum(-1)
                        + k_range * Q.sum(-1, keepdim=True) * K.amax(-1))
    top = ds.masked_fill(~seen, 0.0).amax(-1, keepdim=True)
    z = (s * (q.double() @ k.double().T)).masked_fill(~seen, -float("inf"))
    p = torch.softmax(z, -1)
    pv = p @ V.abs()
    return ref, torch.expm1(2 * top) * pv + 1e-5 * pv + p @ v_error.expand(V.shape)


def check(got, ref, bound):
    err = (got.double() - ref).abs()
    print(f"largest error / bound {float((err / bound).max()):.3f}")
    assert torch.isfinite(got).all() and torch.all(err <= bound)


@pytest.mark.parametrize("hd", [32, 64, 128, 256])
@pytest.mark.parametrize("lift", [0, 15, 20, 26])
def test_prompt_channels(hd, lift):
    n, nq, nkv, s = 600, 4, 2, hd ** -0.5
    q, k, v = normal(15, n, nq, hd), normal(16, n, nkv, hd), normal(17, n, nkv, hd)
    q[..., 3] *= 2.0 ** lift                     # the same products
    k[..., 3] *= 2.0 ** -lift
    q[..., 7] *= 2.0 ** -lift                    # and a key's channel far above its others
    k[..., 7] *= 2.0 ** lift
    v[..., 5] *= 2.0 ** -lift
    got = ops.prompt_attention(q, k, v, [0, n], s)
    seen = forms.causal(n, n)
    for h in range(nq):
        vh = v[:, h // 2]
        v_error = torch.full((1, 1), 2.0 ** -39, device="cuda").double() * vh.abs().max()
        ref, bound = head_bound(q[:, h], k[:, h // 2], vh, seen, s, 2.0 ** -39, v_error)
        check(got[:, h], ref, bound)


@pytest.mark.parametrize("hd", [32, 64, 128, 256])
@pytest.mark.parametrize("lift", [0, 8, 15, 20])
def test_prefix_channels(hd, lift):
    B, nq, nkv, P, s = 5, 4, 2, 2000, hd ** -0.5
    q, kp, vp = normal(18, B, nq, hd), normal(19, nkv, P, hd), normal(20, nkv, P, hd)
    q[..., 3] *= 2.0 ** lift
    kp[..., 3] *= 2.0 ** -lift
    q[..., 7] *= 2.0 ** -lift
    kp[..., 7] *= 2.0 ** lift
    vp[..., 5] *= 2.0 ** -lift
    kp[:, ::50] *= 2.0 ** -9                     # rows that the piece's scale only just fits
    vp[:, ::50] *= 2.0 ** -9
    empty = torch.empty(B, nkv, 1, hd, device="cuda")
    got = ops.prefix_attention(q, kp, vp, P, empty, empty, [0] * B, s)
    seen = torch.ones(B, P, dtype=torch.bool, device="cuda")
    for h in range(nq):
        vh = vp[h // 2]
        v_error = 2.0 ** -22 * vh.double().abs().amax(-1, keepdim=True)
        ref, bound = head_bound(q[:, h], kp[h // 2], vh, seen, s, 2.0 ** -22, v_error)
        check(got[:, h], ref, bound)
