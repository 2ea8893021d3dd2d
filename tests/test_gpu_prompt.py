"""GPU parity of the prompt and batch operators (embed_tokens, qk_norm_rope,
prompt_attention, prefix_attention) with plain 64-bit forms in numpy / torch.

Tolerances, from the arithmetic (u = 2^-24, half a step of f32):
  embed    : a weight is rounded at most once and scaled with one more
             rounding: 2 u |y|, and for Q4_K its fma rounds d*sc*q - dmin*m
             once, relative to the difference; 3 u |y| covers all.
  rotation : the row's norm factor (sum of hd squares: hd u at most, here
             bounded by 16 u for its pairwise sums of 8, a 5-step tree and the
             divide and square root, each a few u), two products: 20 u; the
             angle is off by u pi / 4 + sincospi's 2 u: each of the two
             products of a pair by 4 u; their sum rounds once: together within
             32 u (|a| + |b|) of the pair.
  attention: as test_gpu_attention: |ds| <= (hd + 32) u smax per score, where
             smax = max_t sum_i |scale q k|, twice that in a weight ratio; the
             weights' and the running sums' roundings are O(n u) at worst in
             the length and O(sqrt n u) as they fall; (8 (hd + 32) u smax +
             1e-5) * sum_t p_t |v_t| as there.
"""
import ctypes as C

import numpy as np
import pytest
import torch

import oracle
from quantized_weight_streaming_q4k_gb300 import _lib, build, ops, synth

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
W_PROMPT = 70        # workload id of this file's seeds


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    torch.cuda.set_device(0)
    yield
    assert ops.device_error() == 0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(W_PROMPT * 1000 + seed)
    return g


def normal(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


# ------------------------------------------------------------------ embed
MATRIX = {ops.Q4_0: synth.q4_0_matrix, ops.Q8_0: synth.q8_0_matrix, ops.Q4_K: synth.q4_k_matrix,
          ops.Q6_K: synth.q6_k_matrix}


@pytest.mark.parametrize("fmt", list(MATRIX))
@pytest.mark.parametrize("hidden,n,scale", [(256, 1, 1.0), (2560, 77, 50.596443), (512, 5, -0.37)])
def test_embed_rows(fmt, hidden, n, scale):
    vocab = 301
    g = synth.rng(W_PROMPT, 1, fmt, hidden)
    W = MATRIX[fmt](g, vocab, hidden)
    tok = g.integers(0, vocab, n)
    tok[0], tok[-1] = vocab - 1, 0
    if n > 3:
        tok[1] = tok[2]                                    # the same row twice
    Wd = torch.from_numpy(W).cuda()
    y = ops.embed_tokens(fmt, Wd, torch.from_numpy(tok).cuda(), vocab, hidden, scale)
    rows = oracle.dequant(fmt, W, vocab, hidden)[tok]
    ref = rows * float(np.float32(scale))
    assert np.all(np.abs(y.cpu().numpy().astype(np.float64) - ref) <= 3 * U * np.abs(ref))
    assert torch.equal(y, ops.embed_tokens(fmt, Wd, torch.from_numpy(tok).cuda(), vocab, hidden,
                                           scale))


@pytest.mark.parametrize("fmt,hidden", [(ops.Q4_0, 32), (ops.Q4_0, 96), (ops.Q8_0, 544)])
def test_embed_small_blocks(fmt, hidden):
    g = synth.rng(W_PROMPT, 2, fmt, hidden)
    W = MATRIX[fmt](g, 40, hidden)
    tok = np.arange(40)[::-1].copy()
    y = ops.embed_tokens(fmt, torch.from_numpy(W).cuda(), torch.from_numpy(tok).cuda(), 40, hidden)
    ref = oracle.dequant(fmt, W, 40, hidden)[tok]
    assert np.all(np.abs(y.cpu().numpy().astype(np.float64) - ref) <= 3 * U * np.abs(ref))


def test_embed_token_outside_the_table():
    W = torch.from_numpy(synth.q4_0_matrix(synth.rng(W_PROMPT, 3), 10, 64)).cuda()
    tok = torch.tensor([3, 10, -1, 9], device="cuda")
    y = ops.embed_tokens(ops.Q4_0, W, tok, 10, 64)
    code = C.c_uint(0)
    assert _lib.lib().qws_device_error(C.byref(code)) == 7 and code.value == 512
    assert ops.device_error() == 0                        # read once
    good = ops.embed_tokens(ops.Q4_0, W, torch.tensor([3, 9], device="cuda"), 10, 64)
    assert torch.equal(y[0], good[0]) and torch.equal(y[3], good[1])
    assert not y[1:3].any()



# ------------------------------------------------------------------ qk_norm_rope
def rotate64(x, pos, rot, base, w, eps):
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    half = rot // 2
    f = torch.tensor([base ** (-2.0 * i / rot) for i in range(half)], dtype=torch.float64,
                     device="cuda")
    th = (pos.double()[:, None] * f)[:, None]
    a, b = y[..., :half], y[..., half:rot]
    z = torch.cat([a * th.cos() - b * th.sin(), a * th.sin() + b * th.cos(), y[..., rot:]], -1)
    pair = a.abs() + b.abs()
    return z, torch.cat([pair, pair, y[..., rot:].abs()], -1)


def check_qk(q, k, pos, rot, base, w_q, w_k, got, eps=1e-6):
    for x, w, y in ((q, w_q, got[0]), (k, w_k, got[1])):
        ref, size = rotate64(x, pos, rot, base, w, eps)
        # 2^-40: the reference's own angle (f64 product, far positions)
        assert torch.all((y.double() - ref).abs() <= (32 * U + 2.0 ** -32) * size)


@pytest.mark.parametrize("nq,nkv,hd,rot", [(8, 4, 256, 256), (16, 4, 128, 64), (3, 1, 64, 64),
                                           (4, 4, 32, 32), (6, 2, 128, 20), (8, 8, 64, 2)])
@pytest.mark.parametrize("n", [1, 3, 130])
@pytest.mark.parametrize("norm", [True, False])
def test_qk_norm_rope(nq, nkv, hd, rot, n, norm):
    g = gen(nq * hd + n)
    q, k = normal(g, n, nq, hd), normal(g, n, nkv, hd)
    w_q, w_k = (1 + 0.1 * normal(g, hd), 1 + 0.1 * normal(g, hd)) if norm else (None, None)
    pos = torch.randint(0, 5000, (n,), device="cuda", generator=g)
    got = ops.qk_norm_rope(q, k, pos, rot, 1e4, w_q, w_k)
    check_qk(q, k, pos, rot, 1e4, w_q, w_k, got)
    if not norm:
        assert torch.equal(got[0][..., rot:], q[..., rot:])


@pytest.mark.parametrize("base", [1.0, 500.0, 1e6])
def test_qk_far_positions(base):
    g = gen(1)
    pos = torch.tensor([0, 1, 131071, 1000003, 2 ** 24 + 1, 2 ** 31 - 1, -1, -70000],
                       device="cuda")
    q, k = normal(g, 8, 2, 256), normal(g, 8, 1, 256)
    got = ops.qk_norm_rope(q, k, pos, 256, base)
    for x, y in ((q, got[0]), (k, got[1])):
        ref, size = rotate64(x, pos, 256, base, None, 0.0)
        # the reference's angle is a rounded f64 product: |angle| 2^-52 off
        off = 32 * U + pos.double().abs()[:, None, None] * 2.0 ** -51
        assert torch.all((y.double() - ref).abs() <= off * size)


def test_qk_views_in_place_and_into_a_cache():
    g = gen(2)
    n, nq, nkv, hd, room = 77, 8, 4, 128, 200
    qkv = normal(g, n, nq + 2 * nkv, hd)
    q, k, v = qkv[:, :nq], qkv[:, nq:nq + nkv], qkv[:, nq + nkv:]
    w_q, w_k = 1 + 0.1 * normal(g, hd), 1 + 0.1 * normal(g, hd)
    pos = 50 + torch.arange(n, device="cuda")
    q0, k0, v0 = q.clone(), k.clone(), v.clone()
    plain = ops.qk_norm_rope(q0, k0, pos, hd, 1e4, w_q, w_k)
    # k into rows 50 .. of a cache [n_kv][room][hd]; the rest of it untouched
    cache = torch.full((nkv, room, hd), 7.0, device="cuda")
    into = cache[:, 50:50 + n].transpose(0, 1)
    ops.qk_norm_rope(q, k, pos, hd, 1e4, w_q, w_k, k_out=into)
    assert torch.equal(into, plain[1])
    assert torch.all(cache[:, :50] == 7.0) and torch.all(cache[:, 50 + n:] == 7.0)
    # in place on the fused rows: values keep theirs
    ops.qk_norm_rope(q, k, pos, hd, 1e4, w_q, w_k, q_out=q, k_out=k)
    assert torch.equal(q, plain[0]) and torch.equal(k, plain[1]) and torch.equal(v, v0)


def test_qk_matches_rope_at_pos():
    g = gen(3)
    q, k = normal(g, 1, 8, 256), normal(g, 1, 4, 256)
    pos = torch.tensor([1234], device="cuda")
    a, b = ops.qk_norm_rope(q, k, pos, 128, 1e4)
    ops.rope_at_pos(q[0], 8, 256, 128, 1234, 1e4)
    ops.rope_at_pos(k[0], 4, 256, 128, 1234, 1e4)
    for x, y in ((a[0], q[0]), (b[0], k[0])):
        size = torch.cat([x[..., :64].abs() + x[..., 64:128].abs()] * 2 + [x[..., 128:].abs()], -1)
        assert torch.all((x - y).abs() <= 33 * U * 1.5 * size)


def test_qk_zero_and_huge_heads():
    z = torch.zeros(2, 1, 64, device="cuda")
    pos = torch.arange(2, device="cuda")
    a, _ = ops.qk_norm_rope(z, z, pos, 64, 1e4, torch.ones(64, device="cuda"), None)
    assert not a.any()
    big = torch.full((1, 1, 64), 1e15, device="cuda")
    a, _ = ops.qk_norm_rope(big, big, pos[:1], 64, 1e4, torch.ones(64, device="cuda"), None)
    assert torch.all((a - 1).abs() <= 32 * U)


# ------------------------------------------------------------------ attention, 64 bits
def rows64(q, k, v, seen, scale, cap):
    """(out, tolerance) of rows q [n, hd] over keys k, v [m, hd], seen [n, m]."""
    hd = q.shape[-1]
    kd, vd = k.double(), v.double()
    z = scale * (q.double() @ kd.T)
    size = abs(scale) * (q.double().abs() @ kd.abs().T)
    if cap:
        z = cap * torch.tanh(z / cap)
    z = z.masked_fill(~seen, -float("inf"))
    p = torch.softmax(z, -1).nan_to_num(0.0)
    smax = size.masked_fill(~seen, 0.0).amax(-1, keepdim=True) if k.shape[0] else 0.0
    return p @ vd, (8 * (hd + 32) * U * smax + 1e-5) * (p @ vd.abs())


def check_prompt(q, k, v, cu, out, scale, cap=0.0, ck=None):
    nq, nkv = q.shape[1], k.shape[1]
    ck = cu if ck is None else ck
    for a, b, c, d in zip(cu, cu[1:], ck, ck[1:]):
        i = torch.arange(b - a, device="cuda")[:, None] + (d - c) - (b - a)
        seen = torch.arange(d - c, device="cuda")[None] <= i
        for h in range(nq):
            g = h // (nq // nkv)
            if d == c:
                assert not out[a:b, h].any()
                continue
            ref, tol = rows64(q[a:b, h], k[c:d, g], v[c:d, g], seen, scale, cap)
            err = (out[a:b, h].double() - ref).abs()
            assert torch.all(err <= tol), (a, h, float((err - tol).max()))


def run_prompt(g, lens, nq, nkv, hd, cap=0.0, ctx=None, scale=None, **kw):
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    ck = None if ctx is None else np.concatenate([[0], np.cumsum(ctx)]).tolist()
    tk = cu[-1] if ck is None else ck[-1]
    q, k, v = normal(g, cu[-1], nq, hd), normal(g, tk, nkv, hd), normal(g, tk, nkv, hd)
    scale = hd ** -0.5 if scale is None else scale
    out = ops.prompt_attention(q, k, v, cu, scale, cap, cu_seqlens_k=ck, **kw)
    check_prompt(q, k, v, cu, out, scale, cap, ck)
    assert torch.equal(out, ops.prompt_attention(q, k, v, cu, scale, cap, cu_seqlens_k=ck))
    return q, k, v, cu, out


@pytest.mark.parametrize("n", [1, 2, 15, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300, 1000])
def test_prompt_lengths(n):
    run_prompt(gen(n), [n], 8, 4, 256)


@pytest.mark.parametrize("nq,nkv,hd", [(1, 1, 32), (4, 4, 128), (8, 2, 64), (6, 3, 32), (16, 4, 128),
                                       (3, 1, 256), (2, 1, 64), (4, 1, 256)])
@pytest.mark.parametrize("lens", [[77], [200, 1, 130]])
def test_prompt_head_layouts(nq, nkv, hd, lens):
    run_prompt(gen(nq * hd), lens, nq, nkv, hd)


@pytest.mark.parametrize("cap", [50.0, 1.5])
def test_prompt_softcap(cap):
    run_prompt(gen(11), [190, 65], 8, 4, 128, cap=cap, scale=0.3)


def test_prompt_ragged_with_empty_sequences():
    run_prompt(gen(12), [0, 5, 0, 0, 700, 1, 64, 0, 333, 0], 4, 2, 128)


def test_prompt_many_sequences():
    lens = [(i * 7) % 23 for i in range(300)]             # more than one launch's table
    run_prompt(gen(13), lens, 4, 2, 64)


@pytest.mark.parametrize("lens,ctx", [([1], [1000]), ([64], [1500]), ([100, 3], [611, 3]),
                                      ([5, 200], [2048, 777])])
def test_prompt_continued(lens, ctx):
    run_prompt(gen(14), lens, 8, 4, 256, ctx=ctx)
    run_prompt(gen(15), lens, 4, 1, 64, ctx=ctx)


def test_prompt_rows_without_a_key_are_zero():
    # fewer keys than queries: the first rows see nothing
    q, k, v, cu, out = run_prompt(gen(16), [50, 40, 9], 4, 2, 64, ctx=[20, 0, 9])
    assert not out[:30].any() and not out[50:90].any()
    assert out[30:50].abs().sum(-1).min() > 0


def test_prompt_long_one():
    run_prompt(gen(17), [2500], 4, 2, 128)


def test_prompt_strided_views_and_rows_behind_the_end():
    g = gen(18)
    n, nq, nkv, hd = 150, 8, 4, 64
    qkv = normal(g, n + 9, nq + 2 * nkv, hd)
    q, k, v = qkv[:, :nq], qkv[:, nq:nq + nkv], qkv[:, nq + nkv:]
    wide = torch.full((n + 9, nq + 3, hd), 5.0, device="cuda")
    cu = [4, 70, 150]                                      # rows before and behind: not touched
    out = wide[:, 1:1 + nq]
    got = ops.prompt_attention(q, k, v, cu, 0.125, out=out)
    assert got is out
    check_prompt(q, k, v, cu, out, 0.125)
    assert torch.all(wide[:4] == 5.0) and torch.all(wide[150:] == 5.0)
    assert torch.all(wide[:, 0] == 5.0) and torch.all(wide[:, 1 + nq:] == 5.0)
    # keys and values straight from caches [n_kv][room][hd]
    kc = k.transpose(0, 1).contiguous().transpose(0, 1)
    vc = v.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(ops.prompt_attention(q, kc, vc, cu, 0.125)[4:150], out[4:150])


@pytest.mark.parametrize("hd", [64, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3.0e38])
def test_prompt_masked_places_may_hold_anything(bad, hd):
    g = gen(19)
    n, nq, nkv = 300, 4, 2
    q, k, v = normal(g, n, nq, hd), normal(g, n, nkv, hd), normal(g, n, nkv, hd)
    cu = [0, 100, 230]
    want = ops.prompt_attention(q, k, v, cu, 0.125)
    # behind the last sequence; and the last keys of each, seen by the last rows alone
    k2, v2 = k.clone(), v.clone()
    for t in (k2, v2):
        t[230:] = bad
        t[95:100] = bad
        t[225:230, :, ::3] = bad
    got = ops.prompt_attention(q, k2, v2, cu, 0.125)
    clean = list(range(95)) + list(range(100, 225))
    ref, tol = want[clean].double(), 2e-5
    assert torch.all((got[clean].double() - ref).abs() <= tol)
    assert torch.isfinite(got[clean]).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_prompt_seen_infinities_show(bad):
    # a value that a row sees reaches that row's output, and only its column
    g = gen(20)
    q, k, v = normal(g, 90, 2, 64), normal(g, 90, 1, 64), normal(g, 90, 1, 64)
    want = ops.prompt_attention(q, k, v, [0, 90], 0.125)
    v[40, 0, 5] = bad
    got = ops.prompt_attention(q, k, v, [0, 90], 0.125)
    assert not torch.isfinite(got[40:, :, 5]).any()
    assert torch.isfinite(got[:40]).all()
    keep = [i for i in range(64) if i != 5]
    assert torch.all((got[40:][..., keep] - want[40:][..., keep]).abs() <= 2e-5)
    k[70, 0, 3] = float("nan")
    got = ops.prompt_attention(q, k, v, [0, 90], 0.125)
    assert torch.isnan(got[70:]).all() and torch.isfinite(got[:40]).all()


@pytest.mark.parametrize("mag", [1e-20, 1e-6, 1e4, 1e15])
def test_prompt_magnitudes(mag):
    # values far from 1 in every operand; scores stay of order 1 through scale
    g = gen(21)
    q, k, v = normal(g, 140, 4, 128), normal(g, 140, 2, 128), normal(g, 140, 2, 128)
    s = 128 ** -0.5
    out = ops.prompt_attention(q * mag, k / mag, v * mag, [0, 140], s)
    check_prompt(q * mag, k / mag, v * mag, [0, 140], out, s)


def test_prompt_outlier_tokens():
    # one huge key channel and one huge value row beside ordinary ones
    g = gen(22)
    q, k, v = normal(g, 200, 4, 64), normal(g, 200, 2, 64), normal(g, 200, 2, 64)
    k[..., 7] *= 300.0
    q[..., 7] *= 0.01
    v[33] *= 1e4
    out = ops.prompt_attention(q, k, v, [0, 200], 0.125)
    check_prompt(q, k, v, [0, 200], out, 0.125)


# the same again with enough (query, key) pairs for the tensor cores (over 2^16)
@pytest.mark.parametrize("nq,nkv,hd", [(1, 1, 32), (4, 4, 128), (8, 2, 64), (6, 3, 32), (16, 4, 128),
                                       (3, 1, 256), (2, 1, 64), (4, 1, 256), (3, 1, 128)])
@pytest.mark.parametrize("lens", [[777], [640, 1, 333], [65, 2, 900, 64]])
def test_prompt_large_head_layouts(nq, nkv, hd, lens):
    run_prompt(gen(60 + nq * hd), lens, nq, nkv, hd)


@pytest.mark.parametrize("hd", [32, 128, 256])
@pytest.mark.parametrize("cap,scale", [(50.0, 0.08), (50.0, 1.5), (1.5, 0.3), (0.05, 0.3)])
def test_prompt_large_softcap(cap, scale, hd):
    # scores well within the cap, about it, and far beyond
    run_prompt(gen(61), [700, 65], 8, 4, hd, cap=cap, scale=scale)


@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0])
def test_prompt_large_scales(scale):
    run_prompt(gen(62), [600], 4, 2, 128, scale=scale)


@pytest.mark.parametrize("lens,ctx", [([130], [4000]), ([512, 3], [1111, 3]), ([1, 400], [3000, 777]),
                                      ([300], [2368])])
def test_prompt_large_continued(lens, ctx):
    run_prompt(gen(63), lens, 8, 4, 256, ctx=ctx)
    run_prompt(gen(64), lens, 4, 1, 64, ctx=ctx)


def test_prompt_large_rows_without_a_key_are_zero():
    q, k, v, cu, out = run_prompt(gen(65), [700, 300, 129], 4, 2, 64, ctx=[520, 0, 64])
    assert not out[:180].any() and not out[700:1000].any() and not out[1000:1065].any()
    assert out[180:700].abs().sum(-1).min() > 0


def test_prompt_large_many_sequences():
    lens = [(i * 29) % 97 for i in range(300)]            # more than one launch's table
    run_prompt(gen(66), lens, 4, 2, 64)


def test_prompt_large_strided_views_and_rows_behind_the_end():
    g = gen(67)
    n, nq, nkv, hd = 900, 8, 4, 128
    qkv = normal(g, n + 9, nq + 2 * nkv, hd)
    q, k, v = qkv[:, :nq], qkv[:, nq:nq + nkv], qkv[:, nq + nkv:]
    wide = torch.full((n + 9, nq + 3, hd), 5.0, device="cuda")
    cu = [4, 370, 900]
    out = wide[:, 1:1 + nq]
    assert ops.prompt_attention(q, k, v, cu, 0.09, out=out) is out
    check_prompt(q, k, v, cu, out, 0.09)
    assert torch.all(wide[:4] == 5.0) and torch.all(wide[900:] == 5.0)
    assert torch.all(wide[:, 0] == 5.0) and torch.all(wide[:, 1 + nq:] == 5.0)
    kc = k.transpose(0, 1).contiguous().transpose(0, 1)
    vc = v.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(ops.prompt_attention(q, kc, vc, cu, 0.09)[4:900], out[4:900])
    # one key and value head for all (stride 0)
    k1, v1 = k[:, :1].expand(-1, nkv, -1), v[:, :1].expand(-1, nkv, -1)
    check_prompt(q, k1, v1, cu, ops.prompt_attention(q, k1, v1, cu, 0.09), 0.09)


@pytest.mark.parametrize("hd", [32, 64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3.0e38])
def test_prompt_large_masked_places_may_hold_anything(bad, hd):
    g = gen(68)
    n, nq, nkv = 1100, 4, 2
    q, k, v = normal(g, n, nq, hd), normal(g, n, nkv, hd), normal(g, n, nkv, hd)
    cu = [0, 450, 1000]
    want = ops.prompt_attention(q, k, v, cu, 0.1)
    k2, v2 = k.clone(), v.clone()
    for t in (k2, v2):
        t[1000:] = bad
        t[440:450] = bad
        t[991:1000, :, ::3] = bad
    got = ops.prompt_attention(q, k2, v2, cu, 0.1)
    clean = list(range(440)) + list(range(450, 991))
    assert torch.all((got[clean] - want[clean]).abs() <= 2e-5)


@pytest.mark.parametrize("hd", [64, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_prompt_large_seen_infinities_show(bad, hd):
    g = gen(69)
    q, k, v = normal(g, 700, 2, hd), normal(g, 700, 1, hd), normal(g, 700, 1, hd)
    want = ops.prompt_attention(q, k, v, [0, 700], 0.1)
    v[333, 0, 5] = bad
    got = ops.prompt_attention(q, k, v, [0, 700], 0.1)
    assert not torch.isfinite(got[333:, :, 5]).any()
    assert torch.isfinite(got[:333]).all()
    keep = [i for i in range(hd) if i != 5]
    assert torch.all((got[333:][..., keep] - want[333:][..., keep]).abs() <= 2e-5)
    k[600, 0, 3] = float("nan")
    got = ops.prompt_attention(q, k, v, [0, 700], 0.1)
    assert torch.isnan(got[600:]).all() and torch.isfinite(got[:333]).all()
    q[650, 0, 1] = float("nan")                            # a row's own, and no other row's
    k[600, 0, 3] = v[333, 0, 5] = 0.0
    got = ops.prompt_attention(q, k, v, [0, 700], 0.1)
    assert torch.isnan(got[650, 0]).all()
    got[650, 0] = 0.0
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("hd", [32, 256])
@pytest.mark.parametrize("mag", [1e-20, 1e-6, 1e4, 1e15])
def test_prompt_large_magnitudes(mag, hd):
    g = gen(70)
    q, k, v = normal(g, 640, 4, hd), normal(g, 640, 2, hd), normal(g, 640, 2, hd)
    s = hd ** -0.5
    out = ops.prompt_attention(q * mag, k / mag, v * mag, [0, 640], s)
    check_prompt(q * mag, k / mag, v * mag, [0, 640], out, s)


def test_prompt_large_rows_of_very_different_size():
    g = gen(71)
    q, k, v = normal(g, 800, 4, 64), normal(g, 800, 2, 64), normal(g, 800, 2, 64)
    k[..., 7] *= 300.0
    q[..., 7] *= 0.01
    k[100:110] *= 1e-6
    v[33] *= 1e7
    v[0:3] *= 1e-9                   # the first rows see nothing else
    v[200:205] *= 1e-7
    v[400:440] *= 1e8                # more than half of a tile
    v[640:704] = 0.0
    out = ops.prompt_attention(q, k, v, [0, 800], 0.125)
    check_prompt(q, k, v, [0, 800], out, 0.125)


def test_prompt_large_in_graphs_and_beside_another_call():
    g = gen(72)
    a = [normal(g, 700, h, 256) for h in (8, 4, 4)]
    b = [normal(g, 900, h, 64) for h in (8, 2, 2)]
    want = [ops.prompt_attention(*a, [0, 100, 700], 0.06), ops.prompt_attention(*b, [0, 900], 0.1, 30.0)]
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):                                    # both at once, each its workspace
        with torch.cuda.stream(side[0]):
            outs.append(ops.prompt_attention(*a, [0, 100, 700], 0.06))
        outs.append(ops.prompt_attention(*b, [0, 900], 0.1, 30.0, stream=side[1]))
    torch.cuda.synchronize()
    for i, t in enumerate(outs):
        assert torch.equal(t, want[i % 2]), i
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x = ops.prompt_attention(*a, [0, 100, 700], 0.06)
        y = ops.prompt_attention(*b, [0, 900], 0.1, 30.0)
    a[2].mul_(-2.0)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(x, want[0] * -2.0) and torch.equal(y, want[1])


# ------------------------------------------------------------------ prefix attention
def check_prefix(q, kp, vp, n_prefix, kc, vc, n_ctx, scale, cap, out):
    nq, nkv = q.shape[1], kp.shape[0]
    grp = nq // nkv
    for b, n in enumerate(n_ctx):
        for g in range(nkv):
            k = torch.cat([kp[g, :n_prefix], kc[b, g, :n]])
            v = torch.cat([vp[g, :n_prefix], vc[b, g, :n]])
            rows = q[b, g * grp:(g + 1) * grp]
            got = out[b, g * grp:(g + 1) * grp].double()
            if k.shape[0] == 0:
                assert not got.any()
                continue
            seen = torch.ones(grp, k.shape[0], dtype=torch.bool, device="cuda")
            ref, tol = rows64(rows, k, v, seen, scale, cap)
            assert torch.all((got - ref).abs() <= tol), (b, g, float(((got - ref).abs() - tol).max()))


def run_prefix(g, n_prefix, n_ctx, nq, nkv, hd, cap=0.0, spare=3):
    B, longest = len(n_ctx), max(n_ctx)
    q = normal(g, B, nq, hd)
    kp, vp = normal(g, nkv, n_prefix + spare, hd), normal(g, nkv, n_prefix + spare, hd)
    kc, vc = normal(g, B, nkv, longest + spare, hd), normal(g, B, nkv, longest + spare, hd)
    for t in (kp, vp):                                     # behind the lengths: anything
        t[:, n_prefix:] = float("nan")
    for b, n in enumerate(n_ctx):
        kc[b, :, n:] = float("nan")
        vc[b, :, n:] = float("inf")
    s = hd ** -0.5
    out = ops.prefix_attention(q, kp, vp, n_prefix, kc, vc, n_ctx, s, cap)
    check_prefix(q, kp, vp, n_prefix, kc, vc, n_ctx, s, cap, out)
    assert torch.equal(out, ops.prefix_attention(q, kp, vp, n_prefix, kc, vc, n_ctx, s, cap))
    return q, kp, vp, kc, vc, out


@pytest.mark.parametrize("n_prefix", [0, 1, 31, 32, 33, 64, 127, 129, 1000, 4099])
@pytest.mark.parametrize("batch", [1, 5, 33])
def test_prefix_lengths(n_prefix, batch):
    n_ctx = [(37 * b) % 150 for b in range(batch)]        # 0 among them: that row has none
    run_prefix(gen(30 + batch), n_prefix, n_ctx, 8, 4, 256)


@pytest.mark.parametrize("n_prefix", [0, 1, 33, 64, 65, 130])
@pytest.mark.parametrize("nq,nkv,hd", [(8, 4, 256), (4, 1, 64), (2, 2, 32), (3, 1, 128)])
def test_prefix_short_shared_long_own(n_prefix, nq, nkv, hd):
    run_prefix(gen(37), n_prefix, [0, 1, 400, 31, 32, 33, 257], nq, nkv, hd)


@pytest.mark.parametrize("n_prefix,n_ctx", [(0, [0, 0]), (1, [0]), (5, [0, 3]), (200, [56, 0, 1]),
                                            (256, [0]), (257, [0]), (0, [256, 7]), (0, [257, 7])])
def test_prefix_few_positions(n_prefix, n_ctx):
    # around the border of the one-kernel form, with and without either part
    run_prefix(gen(38), n_prefix, n_ctx, 8, 4, 128)


@pytest.mark.parametrize("hd", [64, 256])
@pytest.mark.parametrize("mag", [1e-20, 1e-6, 1e4, 1e15])
def test_prefix_magnitudes(mag, hd):
    g = gen(39)
    q, kp, vp = normal(g, 5, 4, hd) * mag, normal(g, 2, 900, hd) / mag, normal(g, 2, 900, hd) * mag
    kc, vc = normal(g, 5, 2, 20, hd) / mag, normal(g, 5, 2, 20, hd) * mag
    out = ops.prefix_attention(q, kp, vp, 900, kc, vc, [20, 0, 1, 7, 20], hd ** -0.5)
    check_prefix(q, kp, vp, 900, kc, vc, [20, 0, 1, 7, 20], hd ** -0.5, 0.0, out)


@pytest.mark.parametrize("hd", [64, 256])
def test_prefix_rows_of_very_different_size(hd):
    # key and value rows far from the piece's scale: each still counts with its own bits
    g = gen(41)
    q, kp, vp = normal(g, 3, 4, hd), normal(g, 2, 700, hd), normal(g, 2, 700, hd)
    kp[:, 100:110] *= 1e-6
    kp[:, 300] *= 30.0
    q[..., : hd // 2] *= 0.05
    vp[:, 200:205] *= 1e7
    vp[:, 400:420] *= 1e-9
    vp[:, 650] = 0.0
    vp[0, 0:64] *= 1e-12          # the rows that the scale is taken from
    kc, vc = normal(g, 3, 2, 5, hd), normal(g, 3, 2, 5, hd)
    out = ops.prefix_attention(q, kp, vp, 700, kc, vc, [5, 0, 2], hd ** -0.5)
    check_prefix(q, kp, vp, 700, kc, vc, [5, 0, 2], hd ** -0.5, 0.0, out)


@pytest.mark.parametrize("first", [0.0, 1e-3, 0.02, 60.0])
def test_prefix_first_rows_unlike_the_rest(first):
    # the rows that a piece takes its scale from
    g = gen(44)
    q, kp, vp = normal(g, 3, 4, 128), normal(g, 2, 900, 128), normal(g, 2, 900, 128)
    kp[:, :64] *= first
    vp[:, :64] *= first
    kc, vc = normal(g, 3, 2, 5, 128), normal(g, 3, 2, 5, 128)
    out = ops.prefix_attention(q, kp, vp, 900, kc, vc, [5, 0, 2], 0.09)
    check_prefix(q, kp, vp, 900, kc, vc, [5, 0, 2], 0.09, 0.0, out)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_prefix_seen_infinities_show(bad):
    g = gen(42)
    q, kp, vp = normal(g, 3, 4, 64), normal(g, 2, 700, 64), normal(g, 2, 700, 64)
    kc = normal(g, 3, 2, 5, 64)
    want = ops.prefix_attention(q, kp, vp, 700, kc, kc, [5, 0, 2], 0.125)
    vp[1, 333, 7] = bad
    got = ops.prefix_attention(q, kp, vp, 700, kc, kc, [5, 0, 2], 0.125)
    assert not torch.isfinite(got[:, 2:, 7]).any()
    keep = [i for i in range(64) if i != 7]
    assert torch.all((got[:, 2:][..., keep] - want[:, 2:][..., keep]).abs() <= 2e-5)
    assert torch.all((got[:, :2] - want[:, :2]).abs() <= 2e-5)


@pytest.mark.parametrize("nq,nkv,hd", [(1, 1, 32), (4, 4, 128), (8, 2, 64), (6, 3, 32), (16, 4, 128),
                                       (3, 1, 256), (4, 1, 256)])
def test_prefix_head_layouts(nq, nkv, hd):
    run_prefix(gen(31), 700, [1, 0, 129, 64, 300, 2, 7], nq, nkv, hd)


@pytest.mark.parametrize("cap", [50.0, 1.5])
def test_prefix_softcap(cap):
    run_prefix(gen(32), 500, [100, 20], 8, 4, 128, cap=cap)


def test_prefix_batches():
    run_prefix(gen(33), 90, [b % 5 for b in range(300)], 4, 2, 64)     # more than one launch's
    run_prefix(gen(34), 20000, [3] * 64, 4, 1, 64)
    run_prefix(gen(35), 3000, [1] * 100, 2, 2, 128)


def test_prefix_one_sequence_equals_kv_attention():
    g = gen(36)
    nq, nkv, hd, n = 8, 4, 256, 900
    kc, vc, q = normal(g, nkv, n, hd), normal(g, nkv, n, hd), normal(g, 1, nq, hd)
    want = ops.kv_attention(q[0], kc, vc, nq, nkv, hd, n, n, 0.0625)
    empty = torch.empty(1, nkv, 1, hd, device="cuda")
    a = ops.prefix_attention(q, kc, vc, n, empty, empty, [0], 0.0625)[0]
    b = ops.prefix_attention(q, kc, vc, 0, kc[None], vc[None], [n], 0.0625)[0]
    for x in (a, b):
        assert torch.all((x - want).abs() <= 2e-5)


# ------------------------------------------------------------------ long buffers
def spread(t, dim, room):
    """t in a buffer where neighbours along dim are room elements of t's rows apart."""
    shape = list(t.shape)
    shape[dim] = room
    big = torch.empty(shape, device="cuda", dtype=t.dtype)
    big.narrow(dim, 0, t.shape[dim]).copy_(t)
    return big


def test_offsets_beyond_32_bits():
    # each operator on buffers of 9 to 12 GB, of which little is used: the same bits as compact
    g = gen(46)
    nq, nkv, hd, P = 8, 4, 64, 700
    room = 2 ** 31 // (3 * hd) + 64
    kp = normal(g, nkv, P, hd)
    big = spread(kp, 1, room)
    assert big.stride(0) * 3 > 2 ** 31
    q, own = normal(g, 2, nq, hd), normal(g, 2, nkv, 40, hd)
    want = ops.prefix_attention(q, kp, kp, P, own, own, [40, 9], 0.1)
    assert torch.equal(ops.prefix_attention(q, big, big, P, own, own, [40, 9], 0.1), want)
    qp = normal(g, 600, nq, hd)
    for n in (30, 600):                                    # either form of prompt_attention
        k = kp[:, :n].transpose(0, 1)
        want = ops.prompt_attention(qp[:n], k, k, [0, n], 0.1)
        far = big[:, :n].transpose(0, 1)
        assert torch.equal(ops.prompt_attention(qp[:n], far, far, [0, n], 0.1), want)
    del big, far
    big = spread(own, 2, room // 2)
    want = ops.prefix_attention(q, kp, kp, P, own, own, [40, 9], 0.1)
    assert torch.equal(ops.prefix_attention(q, kp, kp, P, big, big, [40, 9], 0.1), want)
    assert torch.equal(ops.prefix_attention(q, kp, kp, 3, big, big, [40, 9], 0.1),
                       ops.prefix_attention(q, kp, kp, 3, own, own, [40, 9], 0.1))
    del big
    # tokens far apart, in and out
    wide = torch.empty(600, 2 ** 31 // 590 // 64 * 64, device="cuda")
    assert wide.stride(0) * 599 > 2 ** 31
    qw = wide[:, :nq * hd].unflatten(1, (nq, hd))
    ow = wide[:, 1024:1024 + nq * hd].unflatten(1, (nq, hd))
    qw.copy_(qp)
    k = kp[:, :600].transpose(0, 1)
    want = ops.prompt_attention(qp, k, k, [0, 600], 0.1)
    assert torch.equal(ops.prompt_attention(qw, k, k, [0, 600], 0.1, out=ow), want)
    pos = torch.arange(600, device="cuda")
    a, b = ops.qk_norm_rope(qp, k, pos, hd, 1e4)
    c, d = ops.qk_norm_rope(qw, k, pos, hd, 1e4, q_out=ow)
    assert torch.equal(a, c) and torch.equal(b, d)
    del wide, qw, ow, c
    rows = torch.from_numpy(synth.q8_0_matrix(synth.rng(W_PROMPT, 47), 3, 2560)).cuda().view(3, -1)
    table = torch.empty(900000, rows.shape[1], dtype=torch.uint8, device="cuda")
    tok = torch.tensor([5, 800001, 899999], device="cuda")
    table[tok] = rows
    want = ops.embed_tokens(ops.Q8_0, rows, torch.arange(3, device="cuda"), 3, 2560)
    assert torch.equal(ops.embed_tokens(ops.Q8_0, table, tok, 900000, 2560), want)
    del table
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ streams, graphs, refusals
def test_prompt_ops_on_another_stream_and_in_a_graph():
    g = gen(40)
    nq, nkv, hd, n = 8, 4, 128, 333
    q, k, v = normal(g, n, nq, hd), normal(g, n, nkv, hd), normal(g, n, nkv, hd)
    pos = torch.arange(n, device="cuda")
    cu = [0, 100, 333]
    W = torch.from_numpy(synth.q4_k_matrix(synth.rng(W_PROMPT, 41), 50, 256)).cuda()
    tok = torch.arange(20, device="cuda")
    kc, vc = normal(g, 3, nkv, 40, hd), normal(g, 3, nkv, 40, hd)

    def everything(stream=None):
        e = ops.embed_tokens(ops.Q4_K, W, tok, 50, 256, 2.0, stream=stream)
        qr, kr = ops.qk_norm_rope(q, k, pos, hd, 1e4, stream=stream)
        a = ops.prompt_attention(qr, kr, v, cu, 0.09, stream=stream)
        b = ops.prefix_attention(qr[:3], kt, vt, n, kc, vc, [0, 7, 40], 0.09, stream=stream)
        return e, qr, kr, a, b

    kt, vt = k.transpose(0, 1).contiguous(), v.transpose(0, 1).contiguous()
    want = [t.clone() for t in everything()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = everything(side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    # captured and replayed on new values
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = everything()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    q.mul_(0.5), v.mul_(-1.0), vt.mul_(-1.0)
    graph.replay()
    torch.cuda.synchronize()
    want = everything()
    assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_prefix_right_behind_what_makes_its_input():
    # the kernel before is long, leaves most of the GPU free and writes these heads last
    g = gen(43)
    B, nq, nkv, hd, P = 16, 8, 4, 128, 600
    kp, own = normal(g, nkv, P, hd), normal(g, B, nkv, 40, hd)
    src = [(normal(g, B, 1024, hd), normal(g, B, 256, hd)) for _ in range(2)]
    pos = torch.arange(B, device="cuda")
    q, k = torch.empty(B, 1024, hd, device="cuda"), torch.empty(B, 256, hd, device="cuda")
    lens = [33 + b % 8 for b in range(B)]
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    out = torch.empty(B, nq, hd, device="cuda")

    def step(x, wait=False):
        ops.qk_norm_rope(*x, pos, hd, 1e4, q_out=q, k_out=k)
        if wait:
            torch.cuda.synchronize()
        return ops.prefix_attention(q[:, -nq:], kp, kp, P, own, own, lens, 0.09, workspace=ws,
                                    out=out)

    want = [step(x, True).clone() for x in src]
    for i in range(50):
        torch.cuda.synchronize()
        same = torch.equal(step(src[i % 2]), want[i % 2])
        assert same, i


def test_one_workspace_for_calls_in_a_row_and_two_streams():
    g = gen(48)
    ws = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    calls = []
    for i, (n, nq, nkv, hd) in enumerate([(900, 8, 4, 256), (700, 4, 2, 64), (300, 16, 4, 128)]):
        q, k, v = normal(g, n, nq, hd), normal(g, n, nkv, hd), normal(g, n, nkv, hd)
        calls.append(lambda q=q, k=k, v=v, n=n, **kw: ops.prompt_attention(q, k, v, [0, 40, n], 0.1,
                                                                           **kw))
        kp, kc = normal(g, nkv, 2000 + i, hd), normal(g, 6, nkv, 300, hd)
        calls.append(lambda q=q, kp=kp, kc=kc, **kw: ops.prefix_attention(
            q[:6], kp, kp, kp.shape[1], kc, kc, [300, 0, 31, 200, 1, 64], 0.1, 20.0, **kw))
    want = [c().clone() for c in calls]
    torch.cuda.synchronize()
    got = [c(workspace=ws) for _ in range(5) for c in calls]       # nothing waits in between
    torch.cuda.synchronize()
    for i, t in enumerate(got):
        assert torch.equal(t, want[i % len(calls)]), i
    side = [torch.cuda.Stream() for _ in range(2)]
    half = ws.numel() // 2
    got = [c(workspace=ws[i * half:(i + 1) * half], stream=s)
           for _ in range(5) for c in calls for i, s in enumerate(side)]
    torch.cuda.synchronize()
    for i, t in enumerate(got):
        assert torch.equal(t, want[i // 2 % len(calls)]), i


def test_prompt_refusals():
    q = torch.zeros(10, 4, 64, device="cuda")
    k = torch.zeros(10, 2, 64, device="cuda")
    pos = torch.arange(10, device="cuda")
    with pytest.raises(ValueError):
        ops.prompt_attention(q, k, k, [0, 11], 1.0)
    with pytest.raises(ops.QwsError):
        ops.prompt_attention(q, k, k, [0, 6, 5, 10], 1.0)
    with pytest.raises(ops.QwsError):
        ops.prompt_attention(q, k, k, [-1, 10], 1.0)
    with pytest.raises(TypeError):
        ops.prompt_attention(q, k, k, torch.tensor([0, 10], device="cuda"), 1.0)
    with pytest.raises(ops.QwsError):
        ops.prompt_attention(q, k, k, [0, 10], 1.0, out=q)
    with pytest.raises(ops.QwsError):
        ops.prompt_attention(q, k, k, [0, 10], float("nan"))
    with pytest.raises(TypeError):
        ops.prompt_attention(q.half(), k, k, [0, 10], 1.0)
    with pytest.raises(TypeError):
        ops.prompt_attention(q.cpu(), k, k, [0, 10], 1.0)
    with pytest.raises(ValueError):
        ops.prompt_attention(q.transpose(1, 2), k, k, [0, 10], 1.0)
    with pytest.raises(ops.QwsError):                      # one buffer for all rows
        ops.prompt_attention(q, k, k, [0, 10], 1.0, out=q[:1].clone().expand(10, 4, 64))
    with pytest.raises(ops.QwsError):                      # 5 query heads a kv head
        ops.prompt_attention(torch.zeros(10, 5, 64, device="cuda"), k[:, :1], k[:, :1], [0, 10],
                             1.0)
    with pytest.raises(ops.QwsError):
        ops.prompt_attention(q[..., :48].contiguous(), k[..., :48].contiguous(),
                             k[..., :48].contiguous(), [0, 10], 1.0)
    with pytest.raises(ops.QwsError):
        ops.qk_norm_rope(q, k, pos, 65, 1e4)
    with pytest.raises(ops.QwsError):
        ops.qk_norm_rope(q, k, pos, 64, 0.5)
    with pytest.raises(TypeError):
        ops.qk_norm_rope(q, k, pos.int(), 64, 1e4)
    with pytest.raises(ValueError):
        ops.qk_norm_rope(q, k, pos[:9], 64, 1e4)
    with pytest.raises(ops.QwsError):                      # q and k into one buffer
        t = torch.zeros(10, 4, 64, device="cuda")
        ops.qk_norm_rope(q, q.clone(), pos, 64, 1e4, q_out=t, k_out=t)
    kc = torch.zeros(3, 2, 8, 64, device="cuda")
    kp = torch.zeros(2, 8, 64, device="cuda")
    with pytest.raises(ops.QwsError):
        ops.prefix_attention(q[:3], kp, kp, 9, kc, kc, [0, 0, 0], 1.0)
    with pytest.raises(ops.QwsError):
        ops.prefix_attention(q[:3], kp, kp, 8, kc, kc, [0, 9, 0], 1.0)
    with pytest.raises(ops.QwsError):
        ops.prefix_attention(q[:3], kp, kp, -1, kc, kc, [0, 1, 0], 1.0)
    with pytest.raises(ValueError):
        ops.prefix_attention(q[:3], kp, kp, 8, kc, kc, [0, 0], 1.0)
    with pytest.raises(ops.QwsError):
        long = torch.zeros(2, 300, 64, device="cuda")
        ops.prefix_attention(q[:3], long, long, 300, kc, kc, [1, 2, 3], 1.0,
                             workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    W = torch.zeros(10, 18, dtype=torch.uint8, device="cuda")
    with pytest.raises(ops.QwsError):
        ops.embed_tokens(7, W, pos, 10, 32)
    with pytest.raises(ValueError):
        ops.embed_tokens(ops.Q4_0, W, pos, 11, 32)
    with pytest.raises(TypeError):
        ops.embed_tokens(ops.Q4_0, W, pos.int(), 10, 32)
    # nothing to do: nothing launched
    assert ops.embed_tokens(ops.Q4_0, W, pos[:0], 10, 32).shape == (0, 32)
    assert ops.prompt_attention(q[:0], k[:0], k[:0], [0], 1.0).shape == (0, 4, 64)
    assert ops.prompt_attention(q, k, k, [0, 0, 0], 1.0, out=q.clone() + 3).eq(3).all()
    assert ops.prefix_attention(q[:0], kp, kp, 8, kc[:0], kc[:0], [], 1.0).shape == (0, 4, 64)
    assert ops.qk_norm_rope(q[:0], k[:0], pos[:0], 64, 1e4)[0].shape == (0, 4, 64)


# ------------------------------------------------------------------ a run of them together
def test_prompt_then_batched_decode():
    """One attention block over a prompt and then a decode step of a batch that shares it: embed,
    norm, the Q4_K product for Q, K and V, the heads' norm and rotation (k into the cache), the
    prompt's attention; then one more token per sequence against the shared prefix.  Each row
    equals the one-token path of the same operators (kv_attention over one cache)."""
    g = synth.rng(W_PROMPT, 50)
    vocab, hidden, nq, nkv, hd, n, B = 200, 512, 4, 2, 128, 75, 3
    dim = (nq + 2 * nkv) * hd
    E = torch.from_numpy(synth.q6_k_matrix(g, vocab, hidden)).cuda()
    Wqkv = torch.from_numpy(synth.q4_k_matrix(g, dim, hidden)).cuda()
    w_in, w_q, w_k = (torch.from_numpy(synth.norm_weights(g, m)).cuda() for m in (hidden, hd, hd))
    tok = torch.from_numpy(g.integers(0, vocab, n + B)).cuda()
    scale = hd ** -0.5

    def heads(tokens, positions, k_out=None):
        T = tokens.numel()
        h = ops.embed_tokens(ops.Q6_K, E, tokens, vocab, hidden, hidden ** 0.5)
        x = ops.rms_norm(h, w_in, 1e-6, batch=T)
        y = ops.q4k_prefill_matmul(Wqkv, x, dim, hidden, T).view(T, nq + 2 * nkv, hd)
        q, k = ops.qk_norm_rope(y[:, :nq], y[:, nq:nq + nkv], positions, hd, 1e4, w_q, w_k,
                                k_out=k_out)
        return q, k, y[:, nq + nkv:]

    kc = torch.zeros(nkv, n, hd, device="cuda")
    q, k, v = heads(tok[:n], torch.arange(n, device="cuda"), kc.transpose(0, 1))
    vc = v.transpose(0, 1).contiguous()
    out = ops.prompt_attention(q, k, v, [0, n], scale)
    for i in (0, 1, 40, n - 1):
        one = ops.kv_attention(q[i].contiguous(), kc, vc, nq, nkv, hd, n, i + 1, scale)
        assert torch.all((out[i] - one).abs() <= 2e-5 * vc.abs().max())
    # the same prompt in two chunks gives the same rows
    tail = ops.prompt_attention(q[30:], k, v, [0, n - 30], scale, cu_seqlens_k=[0, n])
    assert torch.all((tail - out[30:]).abs() <= 2e-5 * vc.abs().max())
    # decode: B sequences, one own token each, behind the shared prompt
    q1, k1, v1 = heads(tok[n:], torch.full((B,), n, device="cuda"))
    own_k, own_v = k1[:, :, None].contiguous(), v1[:, :, None].contiguous()
    got = ops.prefix_attention(q1, kc, vc, n, own_k, own_v, [1] * B, scale)
    for b in range(B):
        kb, vb = torch.cat([kc, own_k[b]], 1), torch.cat([vc, own_v[b]], 1)
        one = ops.kv_attention(q1[b].contiguous(), kb, vb, nq, nkv, hd, n + 1, n + 1, scale)
        assert torch.all((got[b] - one).abs() <= 2e-5 * vb.abs().max())
