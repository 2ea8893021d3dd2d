"""Numbers beyond 32 bits that the binding hands to a C int: refused, not cut off (no GPU)."""
import pytest
import torch

from paged_forms import Q4_0, Q8_0, slab_bytes
from quantized_weight_streaming_q4k_gb300 import ops

TABLE = torch.zeros(1, 1, dtype=torch.int32)
CPU = -1                                               # a tensor's get_device()


def paged(fmt, shape, hd=64):
    return ops._paged(fmt, torch.empty(shape, dtype=torch.uint8), TABLE, hd, CPU)


@pytest.mark.parametrize("fmt", [Q4_0, Q8_0])
def test_pages_as_they_are(fmt):
    kv = paged(fmt, (3, 2, 4 * slab_bytes(fmt, 64)))
    assert (kv.fmt, kv.page_size, kv.n_kv_heads, kv.n_pages, kv.n_seqs, kv.max_pages) == \
        (fmt, 64, 2, 3, 1, 1)
    assert paged(fmt, (0, 1, 4096 * slab_bytes(fmt, 64))).page_size == 65536


@pytest.mark.parametrize("high", [2 ** 32, -2 ** 32, 2 ** 40])
@pytest.mark.parametrize("fmt", [Q4_0, Q8_0])
def test_formats(fmt, high):
    # the low 32 bits are a format, whose pages would be read beyond these
    assert paged(fmt + high, (1, 1, 16)).fmt == 0


@pytest.mark.parametrize("fmt", [Q4_0, Q8_0])
def test_page_sizes(fmt):
    for slabs in (4097, 2 ** 28 + 1):                  # 2^32 + 16 positions: 16 in 32 bits
        with pytest.raises(ValueError):
            paged(fmt, (0, 1, slabs * slab_bytes(fmt, 64)))


@pytest.mark.gpu
def test_rotations():
    k = torch.zeros(1, 1, 64, device="cuda")
    i = torch.zeros(1, dtype=torch.int64, device="cuda")
    pages = torch.zeros(1, 1, slab_bytes(Q4_0, 64), dtype=torch.uint8, device="cuda")
    for rot in (2 ** 32 + 64, -2 ** 32, 66, -2, 2 ** 40):
        with pytest.raises(ops.QwsError):
            ops.paged_kv_append(Q4_0, pages, TABLE.cuda(), k, k, i, i, rot_dim=rot)
    with pytest.raises(ops.QwsError):
        ops.paged_kv_append(Q4_0 + 2 ** 32, pages, TABLE.cuda(), k, k, i, i)
