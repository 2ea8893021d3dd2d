"""Attention with spare rows in the table, as a server's step has them, and the number of a
sequence's neighbouring tokens said or not."""
import math

import pytest
import torch

from paged_forms import Q4_0, Q8_0, Pool, paged_attend
from test_gpu_paged import check_attention, dev, gen, make_table, normal

pytestmark = pytest.mark.gpu

FORMATS = [Q4_0, Q8_0]


@pytest.fixture(scope="module")
def ops():
    from quantized_weight_streaming_q4k_gb300 import ops
    ops.device_error()
    return ops


def step(fmt, hd, nq, nkv, new, seed, spare=20, mixed=False):
    """Sequences of ragged lengths with `new` neighbouring tokens each at their ends (at any
    positions of theirs when mixed), in rows of a table that has `spare` more of them than tokens."""
    page, lens = 16, [5 + new, 40, 16 + new - 1, 133, 700]
    per = max(lens) // page + 1
    pool = Pool(fmt, 5 * per, nkv, hd, page).randomise(seed, 0.15 if fmt == Q4_0 else 0.01)
    tight = make_table(5, per, 5 * per, seed)
    rows = torch.randperm(5 * new + spare, generator=torch.Generator().manual_seed(seed))[:5]
    wide = torch.full((5 * new + spare, per), -1, dtype=torch.int32, device="cuda")
    wide[rows.cuda()] = tight
    at = [[n - new + i for i in range(new)] for n in lens]
    if mixed:
        at = [[(7 * i + 3 * s) % n for i in range(new)] for s, n in enumerate(lens)]
    pos = dev([p for ps in at for p in ps])
    seq = torch.arange(5, device="cuda").repeat_interleave(new)
    q = normal(gen(seed), 5 * new, nq, hd)
    return pool, (tight, seq), (wide, rows.cuda()[seq]), q, pos


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hd", [32, 64, 128, 256])
@pytest.mark.parametrize("nq,nkv", [(3, 3), (4, 2), (3, 1), (8, 2)])
@pytest.mark.parametrize("new", [1, 2, 3, 5])
def test_spare_rows(ops, fmt, hd, nq, nkv, new):
    """Whatever is said, the rows are right; said as it is, they are those of a table without
    spare rows, bit for bit."""
    pool, (tight, s), (wide, sw), q, pos = step(fmt, hd, nq, nkv, new, hd + new,
                                                mixed=(nq + new) % 2 == 0)
    told = check_attention(ops, pool, wide, q, sw, pos, hd ** -0.5, tokens_per_seq=new)
    ref, spread, top, peak = paged_attend(pool, wide, q, sw, pos, hd ** -0.5)
    bound = (4 * (hd + 32) * 2.0 ** -24 * top + 1e-5)[..., None] * spread + 2.0 ** -36 * peak[..., None]
    for said in (0, 1, 2, 3, 4):           # the bound is that of check_attention
        out = ops.paged_kv_attention(fmt, pool.pages, wide, q, sw, pos, hd ** -0.5,
                                     tokens_per_seq=said)
        assert bool(((out - ref).abs() <= bound + 1e-30).all())
    assert torch.equal(told, ops.paged_kv_attention(fmt, pool.pages, tight, q, s, pos, hd ** -0.5,
                                                    tokens_per_seq=new))
    if new >= 3:                           # four rows an item, unsaid too
        assert torch.equal(told, ops.paged_kv_attention(fmt, pool.pages, tight, q, s, pos, hd ** -0.5))
    assert ops.device_error() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hd,nq", [(64, 1), (64, 2), (128, 1), (256, 2)])
@pytest.mark.parametrize("n", [1024, 1025, 2600])
def test_many_rows_in_a_larger_table(ops, fmt, hd, nq, n):
    """More rows than a launch's list holds, fewer than the table's: pairs of neighbouring tokens of
    a sequence, which the border between launches parts too, and padding."""
    nkv, page, slots = 1, 16, 64
    pool = Pool(fmt, slots, nkv, hd, page).randomise(2, 0.15 if fmt == Q4_0 else 0.01)
    table = dev([[i % slots, (7 * i + 1) % slots, (5 * i + 3) % slots] for i in range(n + 9)], torch.int32)
    i = torch.arange(n, device="cuda")
    seqs = (i + 1) // 2 * 13 % (n + 9)
    pos = i * 29 % 48
    seqs[5::97] = -1
    q = normal(gen(1), n, nq, hd)
    j = torch.arange(48, device="cuda")
    where = table[:, j // page].long()
    k, v = (pool.read(where, (j % page).expand(n + 9, -1), f)[:, :, 0] for f in (False, True))
    z = torch.einsum("thd,tjd->thj", q.double(), k[seqs]) * hd ** -0.5
    z = z.masked_fill(j > pos[:, None, None], -math.inf)
    ref = torch.einsum("thj,tjd->thd", torch.softmax(z, -1), v[seqs])
    ref[seqs < 0] = 0.0
    for said in (0, 1, 2, 3):
        out = ops.paged_kv_attention(fmt, pool.pages, table, q, seqs, pos, hd ** -0.5,
                                     tokens_per_seq=said)
        assert torch.allclose(out.double(), ref, rtol=1e-4, atol=1e-5)
        assert not out[seqs < 0].any() and ops.device_error() == 0


def test_what_is_said_is_checked(ops):
    pool, _, (wide, sw), q, pos = step(Q4_0, 64, 4, 2, 2, 1)
    with pytest.raises(ValueError):
        ops.paged_kv_attention(Q4_0, pool.pages, wide, q, sw, pos, 0.125, tokens_per_seq=-1)
    out = [ops.paged_kv_attention(Q4_0, pool.pages, wide, q, sw, pos, 0.125, tokens_per_seq=t)
           for t in (4, 10, 2 ** 40)]
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
