"""prompt_attention of queries without any keys (empty k and v, which have no address): zeros."""
import pytest
import torch

import attention_forms as forms
from quantized_weight_streaming_q4k_gb300 import build, ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    torch.cuda.set_device(0)
    yield
    assert ops.device_error() == 0


@pytest.mark.parametrize("n", [1, 30, 700, 70000])          # CUDA cores and tensor cores
@pytest.mark.parametrize("hd", [32, 256])
def test_no_keys_at_all(n, hd):
    q = torch.ones(n, 4, hd, device="cuda")
    k = torch.empty(0, 2, hd, device="cuda")
    assert k.data_ptr() == 0
    out = torch.full_like(q, 7.0)
    got = ops.prompt_attention(q, k, k, [0, n - 1, n], 1.0, cu_seqlens_k=[0, 0, 0], out=out)
    assert got is out and not out.any()


def test_sequences_whose_keys_have_no_queries():
    q = torch.ones(40, 4, 64, device="cuda")
    k = torch.ones(50, 2, 64, device="cuda")
    got = ops.prompt_attention(q, k, k, [0, 40, 40], 1.0, cu_seqlens_k=[0, 0, 50])
    assert not got.any()


@pytest.mark.parametrize("last", [600, 0])
def test_a_whole_table_of_sequences_without_keys(last):
    # 128 sequences a launch: the first launch has no keys, the second some
    g = torch.Generator(device="cuda")
    g.manual_seed(86000)
    lens, ctx = [10] * 128 + [600], [0] * 128 + [last]
    q = torch.randn(sum(lens), 4, 64, device="cuda", generator=g)
    k = torch.randn(last, 2, 64, device="cuda", generator=g)
    cu, ck = ([sum(n[:i]) for i in range(len(n) + 1)] for n in (lens, ctx))
    got = ops.prompt_attention(q, k, k, cu, 0.125, cu_seqlens_k=ck)
    assert not got[:1280].any()
    if last:
        # (pieces, and so roundings, go by all lengths of a call: not the bits of a call of its own)
        args = (q[1280:], k, k, [0, 600], [0, 600], 0.125, 0.0)
        ref = forms.prompt_forms(*args, torch.float64)
        forms.assert_as_good_as_f32(got[1280:], forms.prompt_forms(*args, torch.float32), ref)
    else:
        assert not got.any()


def test_offsets_that_decrease_are_refused_without_rows_too():
    q = torch.ones(10, 4, 64, device="cuda")
    with pytest.raises(ops.QwsError):
        ops.prompt_attention(q, q[:, :2], q[:, :2], [0, 5, 0], 1.0)
    with pytest.raises(ops.QwsError):
        ops.prompt_attention(q, q[:, :2], q[:, :2], [3, 3], 1.0, cu_seqlens_k=[2, 1])
    assert ops.prompt_attention(q[:0], q[:0, :2], q[:0, :2], [0, 0], 1.0).shape == (0, 4, 64)
