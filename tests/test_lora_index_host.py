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
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    folder = tmp_path_factory.mktemp("lora_index")
    source, out = folder / "rules.cpp", folder / "rules.so"
    source.write_text(PROGRAM)
    compiler = shutil.which(os.environ.get("CXX", "g++"))
    assert compiler, "no C++ compiler"
    subprocess.run([compiler, "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
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
