"""C-ABI checks of the prompt and batch operators that need no GPU: every call
below is refused, or has nothing to do, before the first CUDA runtime call."""
import ctypes as C

import pytest

from quantized_weight_streaming_q4k_gb300 import _lib, build

OK, NULL, SHAPE, ALIGN, FORMAT, WORKSPACE = 0, 1, 2, 3, 4, 5
A = 0x10000          # 16-byte-aligned fake device addresses (never dereferenced)
B, D, E = 0x20000, 0x30000, 0x40000
Q4_0, Q8_0, Q4_K, Q6_K = 2, 8, 12, 14


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.lib()


def heads(data=A, token=512, head=64):
    return _lib.QwsHeads(data, token, head)


def ints(*v):
    return (C.c_int64 * len(v))(*v)


def test_embed(lib):
    f = lib.qws_embed_tokens
    ok = dict(fmt=Q4_0, W=A, tok=B, out=D, vocab=10, hidden=64, n=4, scale=1.0)

    def call(**kw):
        a = {**ok, **kw}
        return f(a["fmt"], a["W"], a["tok"], a["out"], a["vocab"], a["hidden"], a["n"], a["scale"],
                 None)

    assert call(n=0) == OK
    assert call(fmt=3) == FORMAT
    assert call(W=None) == NULL and call(tok=None) == NULL and call(out=None) == NULL
    assert call(W=A + 8) == ALIGN and call(tok=B + 4) == ALIGN and call(out=D + 4) == ALIGN
    assert call(hidden=48) == SHAPE and call(hidden=0) == SHAPE and call(hidden=-32) == SHAPE
    assert call(fmt=Q4_K, hidden=128) == SHAPE and call(fmt=Q6_K, hidden=64) == SHAPE
    assert call(vocab=0) == SHAPE and call(n=-1) == SHAPE and call(n=2 ** 31) == SHAPE
    assert call(scale=float("inf")) == SHAPE and call(scale=float("nan")) == SHAPE


def test_qk_norm_rope(lib):
    ok = dict(q=heads(A), k=heads(B), qo=heads(D), ko=heads(E), w_q=A, w_k=A, pos=B, n=4, nq=4,
              nkv=2, hd=64, rot=64, base=1e4, eps=1e-6)

    def call(**kw):
        a = {**ok, **kw}
        return lib.qws_qk_norm_rope(
            a["q"], a["k"], a["qo"], a["ko"], a["w_q"], a["w_k"], a["pos"], a["n"], a["nq"],
            a["nkv"], a["hd"], a["rot"], a["base"], a["eps"], None)

    assert call(n=0) == OK
    assert call(n=0, w_q=None, w_k=None) == OK
    assert call(n=0, qo=heads(A), ko=heads(B)) == OK              # in place
    for name in ("q", "k", "qo", "ko"):
        assert call(**{name: None}) == NULL
        assert call(**{name: heads(None)}) == NULL
        assert call(**{name: heads(A + 4)}) == ALIGN
        assert call(**{name: heads(A, 514)}) == ALIGN
        assert call(**{name: heads(A, -512)}) == SHAPE
    assert call(pos=None) == NULL and call(pos=B + 4) == ALIGN
    assert call(w_q=A + 2) == ALIGN
    assert call(hd=48) == SHAPE and call(rot=0) == SHAPE and call(rot=63) == SHAPE
    assert call(rot=66) == SHAPE and call(base=0.9) == SHAPE and call(base=float("inf")) == SHAPE
    assert call(eps=-1.0) == SHAPE and call(eps=float("nan")) == SHAPE
    assert call(nq=5) == SHAPE and call(nq=10) == SHAPE and call(nkv=0) == SHAPE
    assert call(n=-1) == SHAPE and call(n=2 ** 31) == SHAPE
    # outputs whose heads overlap; in place with other strides; shared outputs
    assert call(qo=heads(D, 64, 64)) == SHAPE and call(ko=heads(E, 512, 32)) == SHAPE
    assert call(qo=heads(D, 0, 64)) == SHAPE
    assert call(qo=heads(A, 1024, 64)) == SHAPE
    assert call(ko=heads(D)) == SHAPE and call(qo=heads(B)) == SHAPE and call(ko=heads(A)) == SHAPE
    assert call(n=0, ko=heads(E, 64, 64 * 1000)) == OK            # a cache's view
    assert call(ko=heads(E, 64, 64 * 3)) == SHAPE                 # with room for 3 of 4 tokens


def prompt(lib, q=heads(A), k=heads(B), v=heads(D), out=heads(E), cu=ints(0, 10), ck=None, n=1,
           nq=4, nkv=2, hd=64, scale=1.0, cap=0.0, ws=None, ws_bytes=0):
    return lib.qws_prompt_attention(q, k, v, out, cu, ck, n, nq, nkv, hd, scale, cap, ws, ws_bytes,
                                    None)


def test_prompt_attention(lib):
    assert prompt(lib, cu=ints(0), n=0) == OK
    assert prompt(lib, cu=ints(3, 3, 3), n=2) == OK               # only empty sequences
    for name in ("q", "k", "v", "out"):
        assert prompt(lib, **{name: None}) == NULL
        assert prompt(lib, **{name: heads(None)}) == NULL
        assert prompt(lib, **{name: heads(A + 8)}) == ALIGN
        assert prompt(lib, **{name: heads(0x90000, 513)}) == ALIGN
        assert prompt(lib, **{name: heads(0x90000, -4)}) == SHAPE
    assert prompt(lib, cu=None) == NULL
    assert prompt(lib, n=-1) == SHAPE
    assert prompt(lib, cu=ints(0, 10, 9), n=2) == SHAPE
    assert prompt(lib, cu=ints(-1, 10)) == SHAPE
    assert prompt(lib, cu=ints(0, 2 ** 31)) == SHAPE
    assert prompt(lib, ck=ints(5, 4)) == SHAPE
    assert prompt(lib, nq=5) == SHAPE and prompt(lib, nq=10) == SHAPE and prompt(lib, hd=96) == SHAPE
    assert prompt(lib, scale=float("inf")) == SHAPE and prompt(lib, cap=-1.0) == SHAPE
    assert prompt(lib, cap=float("nan")) == SHAPE
    assert prompt(lib, out=heads(A)) == SHAPE and prompt(lib, out=heads(D)) == SHAPE
    assert prompt(lib, out=heads(E, 0, 64)) == SHAPE
    assert prompt(lib, out=heads(E, 128, 64)) == SHAPE


def test_prompt_workspace(lib):
    f = lib.qws_prompt_attention_workspace_bytes
    assert f(ints(0, 9), None, 0, 4, 2, 64) == 0
    assert f(ints(0, 9, 3), None, 2, 4, 2, 64) == 0
    assert f(ints(0, 9), None, 1, 5, 2, 64) == 0
    need = f(ints(0, 5000), None, 1, 4, 2, 64)
    assert need > 0
    cu = ints(0, 5000)
    assert prompt(lib, cu=cu, ws=None, ws_bytes=0) == WORKSPACE
    assert prompt(lib, cu=cu, ws=A, ws_bytes=1024) == WORKSPACE
    assert prompt(lib, cu=cu, ws=A + 8, ws_bytes=need) == ALIGN


def test_prefix_attention(lib):
    ok = dict(q=heads(A), kp=B, vp=D, max_prefix=1000, n_prefix=1000, kc=B, vc=D, max_seq=50,
              n_ctx=ints(1, 50, 0), out=heads(E), batch=3, nq=4, nkv=2, hd=64, scale=1.0, cap=0.0)

    def call(ws=A, ws_bytes=1 << 40, **kw):
        a = {**ok, **kw}
        return lib.qws_prefix_attention(
            a["q"], a["kp"], a["vp"], a["max_prefix"], a["n_prefix"], a["kc"], a["vc"],
            a["max_seq"], a["n_ctx"], a["out"], a["batch"], a["nq"], a["nkv"], a["hd"], a["scale"],
            a["cap"], ws, ws_bytes, None)

    assert call(batch=0) == OK
    for name in ("q", "out"):
        assert call(**{name: None}) == NULL and call(**{name: heads(A + 4)}) == ALIGN
    for name in ("kp", "vp", "kc", "vc"):
        assert call(**{name: None}) == NULL and call(**{name: A + 8}) == ALIGN
    assert call(n_ctx=None) == NULL
    assert call(n_prefix=1001) == SHAPE and call(n_prefix=-1) == SHAPE
    assert call(max_prefix=2 ** 31, n_prefix=5) == SHAPE and call(max_seq=2 ** 31) == SHAPE
    assert call(n_ctx=ints(1, 51, 0)) == SHAPE and call(n_ctx=ints(1, -1, 0)) == SHAPE
    assert call(batch=-1) == SHAPE
    assert call(nq=5) == SHAPE and call(hd=65) == SHAPE and call(nq=16, nkv=2) == SHAPE
    assert call(scale=float("nan")) == SHAPE and call(cap=-0.5) == SHAPE
    assert call(out=heads(A)) == SHAPE and call(out=heads(E, 64, 64)) == SHAPE
    need = lib.qws_prefix_attention_workspace_bytes(1000, ints(1, 50, 0), 3, 4, 2, 64)
    assert need > 0
    assert call(ws=None, ws_bytes=0) == WORKSPACE and call(ws_bytes=need // 2) == WORKSPACE
    assert call(ws=A + 4) == ALIGN
    assert lib.qws_prefix_attention_workspace_bytes(1000, ints(1, -1), 2, 4, 2, 64) == 0
    # few positions in all: one kernel, no workspace
    assert lib.qws_prefix_attention_workspace_bytes(100, ints(1, 50, 0), 3, 4, 2, 64) == 0


def test_attention_positions_end_at_2_to_the_30(lib):
    # sums of positions are kept in 32 bits on the device
    over = 2 ** 30 + 1
    assert prompt(lib, cu=ints(0, 8), ck=ints(0, over)) == SHAPE
    assert prompt(lib, cu=ints(over - 2, over)) == SHAPE
    f = lib.qws_prefix_attention_workspace_bytes
    assert f(over, ints(0), 1, 4, 2, 64) == 0 and f(0, ints(over), 1, 4, 2, 64) == 0
    assert f(2 ** 30, ints(0), 1, 4, 2, 64) > 0
    call = lib.qws_prefix_attention
    assert call(heads(A), B, D, over, 5, B, D, 50, ints(1), heads(E), 1, 4, 2, 64, 1.0, 0.0, A,
                1 << 40, None) == SHAPE
    assert call(heads(A), B, D, 100, 5, B, D, over, ints(1), heads(E), 1, 4, 2, 64, 1.0, 0.0, A,
                1 << 40, None) == SHAPE


def test_attention_scale_over_softcap_is_finite(lib):
    assert prompt(lib, scale=1.0, cap=1e-39) == SHAPE
    assert prompt(lib, scale=1e20, cap=1e-20) == SHAPE
    assert lib.qws_prefix_attention(heads(A), B, D, 100, 5, B, D, 50, ints(1), heads(E), 1, 4, 2, 64,
                                    1.0, 1e-39, A, 1 << 40, None) == SHAPE
    assert prompt(lib, cu=ints(0, 5000), scale=1.0, cap=1e-20, ws=None, ws_bytes=0) == WORKSPACE
