"""The host's part of a prompt_attention call, weighing piece lengths, stays short whatever the
lengths (no GPU: the workspace's size is asked for, which plans the call).  Times are taken against
those of plain calls, as machines differ."""
import ctypes as C
import itertools
import time

import pytest

from quantized_weight_streaming_q4k_gb300 import _lib, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.lib()


def plan_time(lib, lens, ctx=None):
    q, k = ((C.c_int64 * (len(v) + 1))(0, *itertools.accumulate(v)) for v in (lens, ctx or lens))
    best = 1.0
    for _ in range(40):
        t = time.perf_counter()
        lib.qws_prompt_attention_workspace_bytes(q, k, len(lens), 8, 4, 256)
        best = min(best, time.perf_counter() - t)
    return best


def plans(lib, lens, ctx, than, than_ctx, at_most):
    for _ in range(3):                                     # a busy machine
        a, b = plan_time(lib, lens, ctx), plan_time(lib, than, than_ctx)
        print(f"{a * 1e6:.1f} us, {b * 1e6:.1f} us: {a / b:.1f} times (at most {at_most})")
        if a <= at_most * b:
            return
    raise AssertionError((a, b))


def test_short_prompts_beside_a_long_one(lib):
    # 6.5 times the short ones alone, whose pieces are not weighed; item by item 16 times
    plans(lib, [20] * 4000 + [2000], None, [20] * 4000, None, 10)


def test_one_token_rows_beside_a_chunk(lib):
    # 2.6 times (whose keys are 1024 caches of 40); item by item 8 times
    plans(lib, [1] * 1024 + [512], [40] * 1024 + [8000], [1] * 1024, [40] * 1024, 5)


def test_a_chunk_on_a_very_long_context(lib):
    # about as long as on a short one; with a count for every step of a piece 20 times
    plans(lib, [128], [1 << 24], [512], [8000], 6)


def test_what_is_measured_is_planned_as_it_was(lib):
    # sizes that show the piece lengths: bytes of the packed tiles and of the partial results
    def size(lens, ctx, nq, nkv, hd):
        q, k = ((C.c_int64 * (len(v) + 1))(0, *itertools.accumulate(v)) for v in (lens, ctx or lens))
        return lib.qws_prompt_attention_workspace_bytes(q, k, len(lens), nq, nkv, hd)

    assert size([512], [8000], 8, 4, 256) == 86971392
    assert size([8192], None, 8, 4, 256) == 67248128
    assert size([1, 515, 64, 2, 1300, 129, 37, 256, 777, 63, 1, 900], None, 16, 4, 128) == 18689536
    assert size([1] * 64, [4000] * 64, 16, 4, 128) == 1061351424
    assert size([37], None, 8, 4, 256) == 0
