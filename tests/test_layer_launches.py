"""How the gradient of the rows' sums is split over launches (csrc/mrr_layer.h),
on the host: a launch holds less than 2^32 threads in all, and its grid's
dimensions are numbers of 31 bits."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = """
#include "mrr_layer.h"
extern "C" int waves(int64_t row_bytes) { return mrr::grad_waves(row_bytes); }
extern "C" int at_once(int64_t top_k) { return mrr::grad_choices_at_once(top_k); }
extern "C" int64_t tokens(int64_t row_bytes, int64_t top_k) { return mrr::grad_launch_tokens(row_bytes, top_k); }
"""
MOST_ROW = 65536 * 4


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is not installed")
    out = tmp_path_factory.mktemp("launches") / "launches.so"
    include = [arg for d in ("moe_token_re_amd/csrc", "include") for arg in ("-I", os.path.join(ROOT, d))]
    res = subprocess.run([gxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-x", "c++", "-", *include, "-o", out], input=SOURCE,
                         text=True, capture_output=True)
    assert res.returncode == 0, res.stderr
    lib = ctypes.CDLL(str(out))
    for f, n in ((lib.waves, 1), (lib.at_once, 1), (lib.tokens, 2)):
        f.argtypes, f.restype = [ctypes.c_int64] * n, ctypes.c_int64 if f is lib.tokens else ctypes.c_int
    return lib


@pytest.mark.parametrize("top_k", range(1, 17))
def test_a_launch_holds_less_than_2_to_the_32_threads(split, top_k):
    kinds = set()
    for row in (2, 2048, 2050, 4096, 4098, 4112, 14336, MOST_ROW):
        waves, at_once, tokens = split.waves(row), split.at_once(top_k), split.tokens(row, top_k)
        kinds.add(waves)
        assert waves in (1, 4, 8) and at_once in (1, 2, 4, 6, 8) and at_once * 2 >= top_k
        groups = -(-top_k // at_once)
        assert groups in (1, 2) and (groups == 2) == (top_k > 8)
        assert 1 << 20 <= tokens < 1 << 31 and tokens * 64 * waves * groups < 1 << 32
        # as the loop over launches has it: the most tokens that the checks let through
        most = (2 ** 31 - 2) // top_k
        assert -(-most // tokens) <= 2 ** 31 // tokens + 1
    assert kinds == {1, 4, 8}
