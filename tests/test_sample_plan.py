"""How many CTAs share a row of sample_tokens (host only: the choice is compiled by itself)."""
import os
import subprocess

import pytest

from conftest import ROOT

SOURCE = r"""
#include <cstdio>
#include <cstdlib>
#include "sample_plan.h"
// vocab, rows, then the clusters of 1, 2, .. 16 that run at once
int main(int, char** v) {
  std::printf("%d", qws::sample_cluster_size(std::atoll(v[1]), std::atoll(v[2]),
                                             [&](int i) { return std::atoi(v[2 + i]); }));
}
"""
# a whole GB300; one whose clusters end at 8, at 1; none
WHOLE = [152, 76, 46, 36, 28, 23, 15, 15, 15, 13, 8, 8, 7, 7, 7, 7]
EIGHT = WHOLE[:8] + [0] * 8
ONE = [152] + [0] * 15


@pytest.fixture(scope="module")
def size(tmp_path_factory):
    to = tmp_path_factory.mktemp("plan")
    (to / "plan.cpp").write_text(SOURCE)
    csrc = os.path.join(ROOT, "quantized_weight_streaming_q4k_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-I", csrc, "-o", to / "plan", to / "plan.cpp"], check=True)

    def run(vocab, rows, at_once):
        return int(subprocess.run([to / "plan", str(vocab), str(rows), *map(str, at_once)], check=True,
                                  capture_output=True, text=True).stdout)
    return run


def test_sizes_of_a_whole_device(size):
    assert [size(v, 1, WHOLE) for v in (1, 2047, 4096, 32000, 32768, 262144, 2 ** 19)] == \
        [1, 1, 2, 15, 16, 16, 16]
    assert size(262144, 64, WHOLE) == 6 and size(262144, 9, WHOLE) == 10
    assert size(50257, 9, WHOLE) == 10 and size(32000, 200, WHOLE) == 1


def test_sizes_that_do_not_run_are_not_chosen(size):
    for rows in (1, 2, 9, 64, 1000):
        for vocab in (1, 5000, 32768, 50257, 262144, 344000):
            assert 1 <= size(vocab, rows, EIGHT) <= 8
        assert size(44032, rows, ONE) == 1
    assert size(262144, 1, EIGHT) == 8
    # a hole among the sizes
    assert size(262144, 1, WHOLE[:9] + [0] * 3 + [7, 0, 0, 0]) == 13
    assert size(262144, 64, [0] * 6 + [15] + [0] * 9) == 7


def test_no_size_that_is_large_enough(size):
    assert size(44033, 1, ONE) == 0 and size(2 ** 19, 3, EIGHT) == 0 and size(1, 1, [0] * 16) == 0
    assert size(1, 1, [0] * 3 + [36] + [0] * 12) == 4
