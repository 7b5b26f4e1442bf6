"""Index arithmetic of the packed attention at sizes that no test can hold in
memory: the functions of na_packed.cuh, compiled for the host."""
import ctypes
import os
import random
import re
import subprocess

import pytest

from vision_sliding_window_b200 import build

SOURCE = r"""
#include "na_packed.cuh"
using namespace na2d::packed;
extern "C" int rows(int nq, int pos, int per, int group) { return rows_of_tile(nq, pos, per, group); }
extern "C" int row(int at, int pos, int per, int group) { return row_in_tile(at, pos, per, group); }
extern "C" long long numbers(int nseq, long long total, int mul, int per) { return part_numbers(nseq, total, mul, per); }
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    where = tmp_path_factory.mktemp("index")
    src, lib = where / "index.cu", where / "index.so"
    src.write_text(SOURCE)
    subprocess.run([build.nvcc(), *build.CFLAGS, "-Xcompiler", "-fvisibility=default", "-shared", "-cudart", "static",
                    "-o", str(lib), str(src)], check=True, capture_output=True)
    host = ctypes.CDLL(str(lib))
    host.numbers.restype = ctypes.c_longlong
    host.numbers.argtypes = [ctypes.c_int, ctypes.c_longlong, ctypes.c_int, ctypes.c_int]
    return host


def test_row_tiles_of_sequences_of_any_length(host):
    rnd = random.Random(0)
    for _ in range(2000):
        group = rnd.choice([1, 2, 3, 7, 8, 64, 100, 128])
        per = 128 // group
        nq = rnd.choice([1, per, 2 ** 24, 2 ** 30, rnd.randint(1, 2 ** 30)])
        pos = rnd.choice([0, nq - 1, max(nq - per, 0), rnd.randrange(nq)])
        assert host.rows(nq, pos, per, group) == min(nq - pos, per) * group
        for at in (0, nq, pos, pos + per, max(pos - 1, 0), rnd.randrange(nq + 1)):
            assert host.row(at, pos, per, group) == min(max(at - pos, 0), per) * group


def test_part_numbers_of_large_batches(host):
    assert host.numbers(3, 2 ** 30, 128, 32) == 2 ** 32 + 3


def test_no_position_is_multiplied_before_it_is_cut():
    """In the tensor-core kernels, whose tiles' rows are 32 bits."""
    csrc = os.path.join(os.path.dirname(build.__file__), "csrc")
    for name in ("na_packed_tc.cu", "na_packed_tc_bwd.cu"):
        with open(os.path.join(csrc, name)) as f:
            source = f.read()
        assert not re.findall(r"\((?:sp\.nq|lo|hi|min\(hi[^)]*\)) - pos\w*\) \* p\.group", source), name
