"""The integer arithmetic of calls over the paged cache (csrc/kv_plan.h), compiled for the host: bounds up to the largest
that the entry points accept."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantized_weight_q4_gb300", "csrc")
INT_MAX = 2 ** 31 - 1
MAX_LEN = INT_MAX - 1024
SOURCE = """
#include "kv_plan.h"
extern "C" {
int max_len() { return qmv::kKvMaxLen; }
int rows_bound(long long rows, int max_rows, int max_len) { return qmv::kv_rows_bound(rows, max_rows, max_len); }
int pages_bound(int n, int page) { return qmv::kv_pages_bound(n, page); }
int written_page(int len, int n, int i, int shift) { return qmv::kv_written_page(len, n, i, shift); }
long long segment_chunks(int n_chunks, int n_blocks, int heads) { return qmv::kv_segment_chunks(n_chunks, n_blocks, heads); }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    at = tmp_path_factory.mktemp("kv_plan")
    (at / "plan.cpp").write_text(SOURCE)
    # -fwrapv: an int that overflows wraps, as in the kernels, and the comparisons below see it
    subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-Wall", "-Werror", "-fPIC", "-shared", "-I", CSRC,
                    str(at / "plan.cpp"), "-o", str(at / "plan.so")], check=True)
    lib = ctypes.CDLL(str(at / "plan.so"))
    lib.rows_bound.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_int]
    lib.segment_chunks.restype = ctypes.c_longlong
    return lib


def test_rows_bound(plan):
    assert plan.max_len() == MAX_LEN
    assert plan.rows_bound(5, INT_MAX, 1000) == 5           # a loose bound reaches the launches as the call's rows
    assert plan.rows_bound(INT_MAX, INT_MAX, 1000) == 1000  # or as the longest sequence's tokens
    assert plan.rows_bound(INT_MAX, INT_MAX, MAX_LEN) == MAX_LEN
    assert plan.rows_bound(100, 7, 1000) == 7 and plan.rows_bound(100, 0, 1000) == 0
    assert plan.rows_bound(5, 3, 0) == 1                    # contradictory numbers are still looked at


@pytest.mark.parametrize("shift", [4, 5, 6, 7])
def test_pages_of_rows(plan, shift):
    page = 1 << shift
    for length in [1, 2, page - 1, page, page + 1, 3 * page + 5]:
        for n in range(length + 1):
            want = sorted({t >> shift for t in range(length - n, length)})
            bound = plan.pages_bound(n, page)
            got = [plan.written_page(length, n, i, shift) for i in range(bound + 3)]
            assert got == want + [-1] * (bound + 3 - len(want))
            assert len(want) <= bound


@pytest.mark.parametrize("shift", [4, 7])
@pytest.mark.parametrize("length,n", [(MAX_LEN, MAX_LEN), (MAX_LEN, 1), (MAX_LEN, 5000), (1000, 3)])
def test_pages_at_the_largest_bounds(plan, length, n, shift):
    """Every index that a grid of the largest bound holds: a page of the rows, or -1."""
    page = 1 << shift
    bound = plan.pages_bound(MAX_LEN, page)
    assert MAX_LEN / page <= bound < 2 ** 31 // page + 2
    first, last = (length - n) >> shift, (length - 1) >> shift
    for i in [0, 1, last - first, last - first + 1, bound // 2, bound - 2, bound - 1]:
        got = plan.written_page(length, n, i, shift)
        assert got == (first + i if first + i <= last else -1)
        assert got * page < 2 ** 31


def test_chunks_of_long_prompts(plan):
    """262144 rows over as many tokens, 16 heads a group of 256: 2^13 chunks for each of 2^19 row blocks is not none."""
    assert plan.segment_chunks(2 ** 13, 2 ** 19, 1) == 2 ** 32
    assert plan.segment_chunks(2 ** 26, 2 ** 28, 2) == 2 ** 55
    assert plan.segment_chunks(0, 7, 8) == plan.segment_chunks(7, 0, 8) == 0
