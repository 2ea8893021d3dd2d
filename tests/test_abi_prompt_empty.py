"""qws_prompt_attention without keys, or without queries, up to the first CUDA call (no GPU)."""
import ctypes as C

import pytest

from quantized_weight_streaming_q4k_gb300 import _lib, build

OK, NULL, SHAPE, ALIGN = 0, 1, 2, 3
Q, OUT, NONE = 0x10000, 0x40000, None


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.lib()


def call(lib, q=Q, k=NONE, v=NONE, out=OUT, cu=(0, 10), ck=(0, 0), ws=None):
    h = [_lib.QwsHeads(p, 512, 64) for p in (q, k, v, out)]
    a, b = (C.c_int64 * len(cu))(*cu), (C.c_int64 * len(ck))(*ck)
    return lib.qws_prompt_attention(*h, a, b, len(cu) - 1, 4, 2, 64, 1.0, 0.0, ws, 0, None)


def test_keys_that_are_not_there_have_no_address(lib):
    # the next check refuses each of these: a workspace that is not aligned
    assert call(lib, ws=0x8) == ALIGN
    assert call(lib, cu=(0, 10, 10), ck=(0, 0, 7), ws=0x8) == ALIGN     # keys without queries
    assert call(lib, q=NONE, ws=0x8) == NULL and call(lib, out=NONE, ws=0x8) == NULL
    assert call(lib, ck=(0, 1), ws=0x8) == NULL                        # a key: k and v are needed
    assert call(lib, ck=(0, 1), k=Q, ws=0x8) == NULL
    assert call(lib, cu=(0, 3, 10), ck=(0, 0, 1), ws=0x8) == NULL


def test_no_queries_no_addresses(lib):
    assert call(lib, q=NONE, out=NONE, cu=(0, 0), ck=(0, 0)) == OK
    assert call(lib, q=NONE, out=NONE, cu=(5, 5, 5), ck=(0, 3, 9)) == OK


def test_offsets_are_looked_at_without_queries_too(lib):
    assert call(lib, cu=(0, 5, 0), ck=(0, 0, 0)) == SHAPE
    assert call(lib, cu=(3, 3), ck=(2, 1)) == SHAPE
    assert call(lib, cu=(-1, -1), ck=(0, 0)) == SHAPE
