"""The shorter steps of the same rounding (csrc/mrr_quotient.h), for products
whose quotients need no more: those with a 16-bit factor, and any 32-bit
factors' on their way to e4m3."""
import ctypes
import math
import os
import random
import shutil
import subprocess
from fractions import Fraction

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = """
#include "mrr_quotient.h"
extern "C" float quotient(double p, double most, double full) { return mrr::short_quotient_to_odd(p, most, 1.0 / most, full); }
"""


@pytest.fixture(scope="module")
def quotient(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is not installed")
    out = tmp_path_factory.mktemp("short") / "short.so"
    res = subprocess.run([gxx, "-std=c++17", "-O2", "-shared", "-fPIC", "-x", "c++", "-", "-I",
                          os.path.join(ROOT, "moe_token_re_amd", "csrc"), "-o", out], input=SOURCE, text=True, capture_output=True)
    assert res.returncode == 0, res.stderr
    lib = ctypes.CDLL(str(out))
    lib.quotient.argtypes, lib.quotient.restype = [ctypes.c_double] * 3, ctypes.c_float
    return lib.quotient


def e4m3(v):
    a = abs(v)
    if a == 0:
        return Fraction(0)
    e = math.floor(math.log2(a))
    e += (Fraction(2) ** (e + 1) <= a) - (Fraction(2) ** e > a)
    step = Fraction(2) ** (max(e, -6) - 3)
    return round(v / step) * step


def check(quotient, p, most, full, rounder):
    if 0 < p <= most:
        for sign in (1, -1):
            got = rounder(Fraction(quotient(float(sign * p), float(most), full)))
            assert got == rounder(full * Fraction(sign * p) / most), (p, most, full)


@pytest.mark.parametrize("bits", [(8, 24), (11, 24), (11, 11)])
def test_next_to_whole_numbers(quotient, bits):
    rng = random.Random(bits[0])
    for _ in range(10000):
        a, b = (rng.randrange(1 << (n - 1), 1 << n) for n in bits)
        most, n = a * b, rng.randrange(1, 254)
        for p in {n * most // 254, -(-n * most // 254)}:
            check(quotient, p, most, 127, round)
            check(quotient, p, most << rng.randrange(20), 127, round)


def test_next_to_e4m3_borders(quotient):
    rng = random.Random(7)
    close = 0
    for _ in range(20000):
        most = rng.randrange(1 << 23, 1 << 24) * rng.randrange(1 << 23, 1 << 24)
        n, shift = rng.randrange(16, 32), rng.randrange(20)  # n / 2^(shift) of 28, to 448: values and what is between
        for p in {n * most // 28, -(-n * most // 28)}:
            p = Fraction(p, 1 << shift)
            if p <= most and p.numerator < 1 << 48:
                off = abs(28 * p * (1 << shift) / most - n) / n
                close += 0 < off < Fraction(1, 1 << 50)
                check(quotient, p, most, 448, e4m3)
    assert close > 20
