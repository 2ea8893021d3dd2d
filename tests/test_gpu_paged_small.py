"""Norms of heads whose squares leave f32's range, with an eps as small or none."""
import pytest
import torch

from paged_forms import Q4_0, Q8_0, Pool, turned

pytestmark = pytest.mark.gpu

SIZES = [1e-10, 2.0 ** -44, 2.0 ** -45, 2.0 ** -46, 1e-15, 1e-18, 1e-20, 1e-22, 1e-25, 1e-38, 1e-40,
         3e-44, 1e15]


@pytest.fixture(scope="module")
def ops():
    from quantized_weight_streaming_q4k_gb300 import ops
    ops.device_error()
    return ops


@pytest.mark.parametrize("fmt", [Q4_0, Q8_0])
@pytest.mark.parametrize("hd,rot", [(32, 32), (64, 64), (128, 50), (256, 256), (256, 0)])
@pytest.mark.parametrize("eps", [0.0, 1e-27, 1e-30, 1e-42, 1e-60, 1e-95])
def test_small_heads(ops, fmt, hd, rot, eps):
    """Every byte of the keys; queries within the bound of f32, 14 u of |a cos| + |b sin|, each at
    most the head's largest before the turn, as for heads of ordinary size."""
    g = torch.Generator(device="cuda")
    g.manual_seed(hd + rot)
    n, nkv = len(SIZES), 3
    size = torch.tensor(SIZES, dtype=torch.float64, device="cuda")[:, None, None]
    k = (torch.randn(n, nkv, hd, device="cuda", generator=g).double() * size).float()
    q = (torch.randn(n, 2 * nkv, hd, device="cuda", generator=g).double() * size).float()
    k[:, 1, 3] *= 64.0                                 # one value far above the others
    k[:, 2, ::2] = 0.0
    v = torch.randn(n, nkv, hd, device="cuda", generator=g)
    w_q, w_k = (1 + 0.1 * torch.randn(hd, device="cuda", generator=g) for _ in range(2))
    pos = torch.arange(n, device="cuda") * 3
    pool, model = (Pool(fmt, 4, nkv, hd, 16) for _ in range(2))
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device="cuda")
    got = ops.paged_kv_append(fmt, pool.pages, table, k, v, torch.zeros_like(pos), pos, rot_dim=rot,
                              base=1e4, w_k=w_k, eps=eps, q=q, w_q=w_q)
    keys = turned(k, w_k, pos, rot, 1e4, eps).float()
    model.write(table[0, pos // 16].long(), pos % 16, keys, v)
    assert torch.equal(pool.pages, model.pages)
    want = turned(q, w_q, pos, rot, 1e4, eps)
    top = turned(q, w_q, pos, 0, 1e4, eps).abs().amax(-1, keepdim=True)
    # (and half a step of the smallest subnormal where a result is one, for each of five roundings)
    assert bool(((got - want).abs() <= 28 * 2.0 ** -24 * top + 5 * 2.0 ** -150).all())
    assert ops.device_error() == 0


@pytest.mark.parametrize("eps", [0.0, 1e-300, 1e-100, 1e-45, 1e-6])
def test_heads_of_zeros(ops, eps):
    hd, nkv = 64, 2
    z = torch.zeros(5, nkv, hd, device="cuda")
    w = torch.full((hd,), 3.0, device="cuda")
    pos = torch.arange(5, device="cuda")
    pool, model = (Pool(Q8_0, 1, nkv, hd, 16, fill=0x5A) for _ in range(2))
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    q = ops.paged_kv_append(Q8_0, pool.pages, table, z, z + 1, torch.zeros_like(pos), pos, rot_dim=hd,
                            w_k=w, eps=eps, q=z, w_q=w)
    model.write(torch.zeros_like(pos), pos, z, z + 1)
    assert torch.equal(pool.pages, model.pages) and not q.any()


def test_an_eps_beyond_the_range_is_refused(ops):
    k = torch.ones(1, 1, 64, device="cuda")
    i = torch.zeros(1, dtype=torch.int64, device="cuda")
    pool = Pool(Q4_0, 1, 1, 64, 16)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    for eps in (2.0 ** 100, 1e39, 1e300, float("inf")):
        with pytest.raises(ops.QwsError):
            ops.paged_kv_append(Q4_0, pool.pages, table, k, k, i, i, eps=eps)
    ops.paged_kv_append(Q4_0, pool.pages, table, k, k, i, i, eps=1e30, w_k=k[0, 0])
    assert ops.device_error() == 0
