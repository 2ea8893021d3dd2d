"""Two tokens of an append with one place in the pages: what is promised of it, and that nothing else
is touched."""
import pytest
import torch

from paged_forms import Q4_0, Q8_0, Pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from quantized_weight_streaming_q4k_gb300 import ops
    ops.device_error()
    return ops


@pytest.mark.parametrize("fmt", [Q4_0, Q8_0])
@pytest.mark.parametrize("hd", [32, 256])
@pytest.mark.parametrize("shared", [False, True])
def test_one_place_for_two_tokens(ops, fmt, hd, shared):
    """The same position twice, or that of another sequence with the same page."""
    nkv, page, n = 3, 16, 300
    g = torch.Generator(device="cuda")
    g.manual_seed(hd)
    table = torch.tensor([[1, 2], [1, 0]], dtype=torch.int32, device="cuda")
    pos = torch.arange(n, device="cuda") % 10                      # 30 tokens each
    seqs = torch.arange(n, device="cuda") // 10 % 2 if shared else torch.zeros_like(pos)
    k, v = (torch.randn(n, nkv, hd, device="cuda", generator=g) for _ in range(2))
    # equal rows: those rows
    pool, model = (Pool(fmt, 3, nkv, hd, page, fill=0xA5) for _ in range(2))
    same = k[:10].repeat(n // 10, 1, 1), v[:10].repeat(n // 10, 1, 1)
    ops.paged_kv_append(fmt, pool.pages, table, *same, seqs, pos)
    at = torch.arange(10, device="cuda")
    model.write(torch.ones_like(at), at, k[:10], v[:10])
    assert torch.equal(pool.pages, model.pages)
    # others: every two bytes are those of one of them, and no others are written
    seen = []
    for i in range(0, n, 10):
        one = Pool(fmt, 3, nkv, hd, page, fill=0xA5)
        one.write(torch.ones_like(at), at, k[i:i + 10], v[i:i + 10])
        seen.append(one.pages.view(torch.int16))
    for _ in range(3):
        got = Pool(fmt, 3, nkv, hd, page, fill=0xA5)
        ops.paged_kv_append(fmt, got.pages, table, k, v, seqs, pos)
        assert bool((torch.stack(seen) == got.pages.view(torch.int16)).any(0).all())
    assert ops.device_error() == 0
