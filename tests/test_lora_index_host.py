"""The index rules of the adapters' kernels (csrc/nf4_lora_index.h), compiled for the host and asked over all sizes: no access
outside the caller's arrays."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "nf4_lora_index.h"
extern "C" int lane_in_row(int values, int t, int rank) { return nf4::lane_in_row(values, t, rank); }
extern "C" int whole_blocks(int first, int N, int blocks) { return nf4::whole_blocks(first, N, blocks); }
extern "C" int column_there(int from, int more, int N) { return nf4::column_there(from, more, N); }
extern "C" int chunk_in_lists(int adapter, int first, int tokens, int most, long long adapters, int listed) {
    return nf4::chunk_in_lists(adapter, first, tokens, most, adapters, listed);
}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    folder = tmp_path_factory.mktemp("lora_index")
    source, out = folder / "rules.cpp", folder / "rules.so"
    source.write_text(PROGRAM)
    compiler = shutil.which(os.environ.get("CXX", "g++"))
    assert compiler, "no C++ compiler"
    subprocess.run([compiler, "-std=c++17", "-O1", "-Wall", "-Werror", "-ftrapv", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "nf4_weight_only_gb300", "csrc"), str(source), "-o", str(out)], check=True)
    return ctypes.CDLL(str(out))


def test_lanes_that_start_in_a_row(rules):
    """What a lane fetches ahead is in its row, and every value of a row is some lane's: the last row of the last adapter
    ends where B ends."""
    for rank in range(8, 129, 8):
        values = 4 if rank <= 16 else 8  # of a lane at a time, as the kernels take them
        starts = [values * t for t in range(4) if rules.lane_in_row(values, t, rank)]
        assert starts and max(starts) + values <= rank
        covered = {s + step + i for s in starts for step in range(0, rank, 4 * values) for i in range(values)
                   if s + step < rank}
        assert covered == set(range(rank))


@pytest.mark.parametrize("n", [1, 8, 255, 256, 257, 511, 512, 513, 5000, (1 << 31) - 513, (1 << 31) - 512, (1 << 31) - 257,
                               (1 << 31) - 256, (1 << 31) - 255, (1 << 31) - 8, (1 << 31) - 1])
def test_blocks_and_columns_up_to_the_widest(rules, n):
    """Python's integers do not overflow; the last blocks of the widest projections end past 2^31."""
    last = (n + 255) // 256 * 256 - 256
    for first in range(max(0, last - 2048), last + 1, 256):
        for blocks in (1, 2):
            assert rules.whole_blocks(first, n, blocks) == (first + 256 * blocks <= n)
        for inside in range(0, 256, 8):
            for more in range(0, 8 * 256, 256):
                assert rules.column_there(first + inside, more, n) == (first + inside + more < n)
    # a lane's column in a block that the row ends inside, as far as 2^31 - 1 reaches
    assert not rules.column_there(min(n + 255, (1 << 31) - 1), 0, n)


def test_chunks_of_any_words(rules):
    """A plan's words may be anything: what passes is inside the order's tokens and the loaded adapters."""
    words = [0, 1, 2, 16, 17, 63, 64, 65, 100, 1 << 24, (1 << 31) - 65, (1 << 31) - 64, (1 << 31) - 2, (1 << 31) - 1, -1, -64,
             -(1 << 31)]
    for adapter in (0, 2, 3, (1 << 31) - 1, -1):
        for first in words:
            for tokens in words:
                for most, listed in ((16, 0), (16, 100), (64, 100), (64, 1 << 24)):
                    inside = 0 <= adapter < 3 and first >= 0 and 1 <= tokens <= most and first + tokens <= listed
                    got = rules.chunk_in_lists(adapter, first, tokens, most, ctypes.c_longlong(3), listed)
                    assert bool(got) == inside, (adapter, first, tokens, most, listed)
