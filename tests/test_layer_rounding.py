"""The steps by which the norm rounds a quotient of 64-bit products to 8 bits
(csrc/mrr_quotient.h), compiled for the host, against exact fractions."""
import ctypes
import math
import os
import random
import shutil
import struct
import subprocess
from fractions import Fraction

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = """
#include "mrr_quotient.h"
extern "C" float quotient(double p, double most, double full) { return mrr::quotient_to_odd(p, most, 1.0 / most, full); }
extern "C" float odd(double d) { return mrr::to_odd(d); }
"""


@pytest.fixture(scope="module")
def steps(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is not installed")
    out = tmp_path_factory.mktemp("quotient") / "quotient.so"
    res = subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC", "-x", "c++", "-", "-I",
                          os.path.join(ROOT, "moe_token_re_amd", "csrc"), "-o", out], input=SOURCE, text=True, capture_output=True)
    assert res.returncode == 0, res.stderr
    lib = ctypes.CDLL(str(out))
    for f, n in ((lib.quotient, 3), (lib.odd, 1)):
        f.argtypes, f.restype = [ctypes.c_double] * n, ctypes.c_float
    return lib


def e4m3(v):
    a = abs(v)
    if a == 0:
        return Fraction(0)
    e = math.floor(math.log2(a))
    e += (Fraction(2) ** (e + 1) <= a) - (Fraction(2) ** e > a)
    step = Fraction(2) ** (max(e, -6) - 3)
    return round(v / step) * step  # to even


def check(steps, p, most):
    for full, rounder in ((127, round), (448, e4m3)):
        exact = full * Fraction(p) / Fraction(most)
        assert rounder(Fraction(steps.quotient(p, most, full))) == rounder(exact), (p.hex(), most.hex(), full)


def f32(rng, lo=-100, hi=100):
    return math.ldexp(rng.randrange(1 << 23, 1 << 24), rng.randrange(lo, hi) - 24) * rng.choice((1, -1))


def test_halves_of_the_largest_and_other_ties(steps):
    """(k + 0.5) / 127 of the largest product, exactly: of all the values 2 p, p, p / 2 ... and of odd parts."""
    rng = random.Random(1)
    check(steps, 1.6515929698944092 / 2 * 1.6830850839614868, 1.6515929698944092 * 1.6830850839614868)
    for _ in range(4000):
        s, w = f32(rng), f32(rng)
        for by in (0.5, 0.25, 1.0, -0.5):
            check(steps, by * s * w, abs(s * w))
        u, k = rng.randrange(1, 1 << 16), rng.randrange(127)
        check(steps, (2 * k + 1) * u * w, abs(254 * u * w))
        k = rng.randrange(1, 448)  # e4m3 values and what is between them
        check(steps, k * u * w, abs(448 * u * w))
        check(steps, (2 * k + 1) * u * w, abs(896 * u * w))


def test_next_to_a_border(steps):
    """Products of 48 bits whose quotient lies off a border by less than 64 bits hold."""
    rng = random.Random(2)
    close = 0
    for _ in range(20000):
        most = rng.randrange(1 << 23, 1 << 24) * rng.randrange(1 << 23, 1 << 24)
        n = 2 * rng.randrange(127) + 1
        for p in {n * most // 254, -(-n * most // 254)}:
            if 0 < p <= most:
                off = abs(Fraction(127 * p, most) - Fraction(n, 2)) / Fraction(n, 2)
                close += 0 < off < Fraction(1, 1 << 54)
                check(steps, float(p), float(most))
                check(steps, -float(p), float(most))
    assert close > 20  # one in some hundreds: 254 p and n most then differ by less than n most 2^-54, a few units


def test_any_products(steps):
    rng = random.Random(3)
    check(steps, 0.0, 1.0)
    for _ in range(20000):
        most, p = abs(f32(rng) * f32(rng)), f32(rng) * f32(rng)
        p = math.ldexp(p, math.frexp(most)[1] - math.frexp(p)[1] - rng.randrange(14))
        if abs(p) <= most:
            check(steps, p, most)


def test_to_odd_keeps_the_side(steps):
    rng = random.Random(4)
    for _ in range(20000):
        d = math.ldexp(rng.random() + 1, rng.randrange(-160, 127)) * rng.choice((1, -1))
        f = steps.odd(d)
        bits = struct.unpack("<I", struct.pack("<f", f))[0]
        if Fraction(f) == Fraction(d):
            continue
        assert bits & 1 and abs(Fraction(f) - Fraction(d)) < Fraction(2) ** max(math.frexp(d)[1] - 24, -149)
    assert steps.odd(0.0) == 0.0 and steps.odd(1.5) == 1.5 and steps.odd(1e300) == math.inf
