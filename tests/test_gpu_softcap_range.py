"""The softcap of the prompt and prefix attention over the whole range of its argument: far above
the scores it changes nothing, far below them every score is +- the cap."""
import pytest
import torch

import attention_forms as forms
from quantized_weight_streaming_q4k_gb300 import build, ops

pytestmark = pytest.mark.gpu
CAPS = [1e20, 1e32, 1e34, 1e36, 1e38, 2.4e38, 3.4e38]


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    torch.cuda.set_device(0)
    yield
    assert ops.device_error() == 0


def normal(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(81000 + seed)
    return torch.randn(shape, device="cuda", generator=g)


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("n,hd", [(30, 64), (700, 64), (700, 256)])      # either form
def test_prompt_cap_far_above_the_scores(n, hd, cap):
    q, k, v = normal(1, n, 4, hd), normal(2, n, 2, hd), normal(3, n, 2, hd)
    cu, s = [0, 11, n], hd ** -0.5
    got = ops.prompt_attention(q, k, v, cu, s, cap)
    ref = forms.prompt_forms(q, k, v, cu, cu, s, cap, torch.float64)
    plain = forms.prompt_forms(q, k, v, cu, cu, s, 0.0, torch.float32)
    forms.assert_as_good_as_f32(got, plain, ref)


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("n_prefix", [40, 700])
def test_prefix_cap_far_above_the_scores(n_prefix, cap):
    nkv, hd, n_ctx = 2, 128, [5, 0, 40]
    q, kp, vp = normal(4, 3, 4, hd), normal(5, nkv, n_prefix, hd), normal(6, nkv, n_prefix, hd)
    kc, vc = normal(7, 3, nkv, 40, hd), normal(8, 3, nkv, 40, hd)
    got = ops.prefix_attention(q, kp, vp, n_prefix, kc, vc, n_ctx, 0.09, cap)
    args = (q, kp, vp, n_prefix, kc, vc, n_ctx, 0.09)
    ref = forms.prefix_forms(*args, cap, torch.float64)
    forms.assert_as_good_as_f32(got, forms.prefix_forms(*args, 0.0, torch.float32), ref)


@pytest.mark.parametrize("cap", [1e-4, 1e-20, 1e-37])
@pytest.mark.parametrize("n", [30, 700])
def test_prompt_cap_far_below_the_scores(n, cap):
    # every weight is e^(+-cap), one to 1e-4 at most: the mean of the visible values
    q, k, v = normal(9, n, 4, 64), normal(10, n, 2, 64), normal(11, n, 2, 64)
    got = ops.prompt_attention(q, k, v, [0, n], 0.125, cap)
    ref = forms.prompt_forms(q, k, v, [0, n], [0, n], 0.125, cap, torch.float64)
    plain = forms.prompt_forms(q, k, v, [0, n], [0, n], 0.0, 0.0, torch.float32)
    mean = forms.prompt_forms(q, k, v, [0, n], [0, n], 0.0, 0.0, torch.float64)
    # the error of a plain mean in f32, and of weights that are off by 2^-22 each
    tol = forms.FACTOR * forms.errors(plain, mean)[1] + 2.0 ** -20 * float(v.abs().max())
    assert forms.errors(got, ref)[1] <= tol


@pytest.mark.parametrize("cap", [0.5, 50.0])
@pytest.mark.parametrize("n,hd", [(700, 32), (700, 128), (700, 256)])
def test_prompt_infinite_scores_reach_the_cap(n, hd, cap):
    # products beyond f32: the cap, not NaN
    q, k, v = normal(12, n, 4, hd), normal(13, n, 2, hd), normal(14, n, 2, hd)
    q[300] *= 1e30
    k[:, :, 0] = 1e18                            # the sign of q's first value decides for all keys
    q[300, :, 1:] = 0.0
    got = ops.prompt_attention(q, k, v, [0, n], 1.0, cap)
    mean = v[:301].double().mean(0).repeat_interleave(2, 0)
    assert torch.all((got[300].double() - mean).abs() <= 301 * 2.0 ** -22 * v[:301].abs().max())
