"""The 8-bit cache's scale is the largest magnitude times the f32 nearest 1 / 127, written out in
numpy on the CPU (a tensor divided by a number is a product on a GPU and a quotient on a CPU)."""
import numpy as np
import pytest
import torch

from paged_forms import Q8_0, Pool

f32 = np.float32
C = f32(1) / f32(127)


def held(x, quotient=False):
    """Codes about zero and f16 scales of blocks x [.., 32]."""
    amax = np.abs(x).max(-1, keepdims=True)
    d = amax / f32(127) if quotient else amax * C
    with np.errstate(divide="ignore"):
        z = np.clip(x * np.where(d == 0, f32(0), f32(1) / d), f32(-127), f32(127))
    code = np.floor(np.abs(z))
    code = np.where(np.abs(z) - code >= 0.5, code + 1, code) * np.sign(z)
    return code, d.astype(np.float16)


def blocks(shape):
    """Blocks [.., 32] of normal values, in every other one halves of a step, which the last bit of a
    scale sends up or down."""
    g = np.random.default_rng(2)
    x = g.standard_normal((*shape, 32)).astype(f32)
    halves = (g.integers(-126, 126, x.shape) + 0.5).astype(f32) * (x[..., :1] / f32(127))
    halves[..., 0] = x[..., 0]
    x[1::2] = halves[1::2]
    return x


def test_the_product_is_not_the_quotient():
    """Rounded once each they differ by a step for some magnitudes, and so do codes, or the choice
    says nothing."""
    x = blocks((2048, 16))
    a = np.abs(x).max(-1)
    assert C == f32(1 / 127) and 0.01 < np.mean(a * C != a / f32(127)) < 0.9
    assert np.sum(held(x)[0] != held(x, True)[0]) > 1000


@pytest.mark.gpu
def test_every_value_held():
    from quantized_weight_streaming_q4k_gb300 import ops
    ops.device_error()
    n, nkv, hd, page = 2048, 2, 256, 64
    x = blocks((2 * n, nkv, hd // 32)).reshape(2, n, nkv, hd)
    x[:, :40] *= f32(2) ** np.arange(-20, 20, dtype=f32)[:, None, None]
    k, v = torch.from_numpy(x).cuda()
    pool = Pool(Q8_0, n // page, nkv, hd, page)
    table = torch.arange(n // page, dtype=torch.int32, device="cuda")[None]
    pos = torch.arange(n, device="cuda")
    seqs = torch.zeros_like(pos)
    ops.paged_kv_append(Q8_0, pool.pages, table, k, v, seqs, pos)
    code, d = held(x.reshape(2, n, nkv, hd // 32, 32))
    want = torch.from_numpy((code * d.astype(f32)).astype(f32).reshape(x.shape)).cuda()
    for out, w, values in zip(ops.paged_kv_gather(Q8_0, pool.pages, table, seqs, pos, hd), want,
                              (False, True)):
        assert torch.equal(out, w)
        assert torch.equal(pool.read(pos // page, pos % page, values), w.double())
    assert ops.device_error() == 0
