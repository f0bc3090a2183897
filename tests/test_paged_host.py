"""Host code of the decode-step entry points.  Runs without a GPU."""
import ctypes as C
import subprocess
from fractions import Fraction

import numpy as np
import pytest

from position_invariant_kv_chunk_gb300 import build as B

# pi to 100 decimals
PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170679,
              10 ** 100)


# ------------------------------------------------------------------- phases --
@pytest.fixture(scope="module")
def turn_fraction(tmp_path_factory):
    d = tmp_path_factory.mktemp("turn")
    (d / "t.cpp").write_text('#include "kamera_hostcheck.h"\n'
                             'extern "C" unsigned long long turn(double x) { return kamera::turn_fraction(x); }\n')
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-I", B.INCLUDE, "-I", B.CSRC, str(d / "t.cpp"),
                    "-o", str(d / "t.so")], check=True)
    f = C.CDLL(str(d / "t.so")).turn
    f.restype, f.argtypes = C.c_ulonglong, [C.c_double]
    return f


@pytest.mark.parametrize("sign", [1, -1])
def test_turn_fraction_is_the_nearest_one(turn_fraction, sign):
    """theta / 2 pi modulo 1 in units of 2^-64: half a unit from the rounding to an
    integer, and the double-double quotient's own error, (2^-53)^2 of the quotient in
    each of three roundings, which is below 2^-30 units for |theta| < 1e4."""
    thetas = [0.0, 0.3, 7.5, 2.5e3, 6.283185307179586, 1e-9, 1e-17, 3e-20, 2.0 ** -60, 0.5, 9999.75]
    thetas += list(1e4 ** (-2.0 * np.arange(32) / 64)) + list(1e6 ** (-2.0 * np.arange(64) / 128))
    one = 2 ** 64
    for t in thetas:
        t = sign * float(t)
        off = (Fraction(turn_fraction(t)) - Fraction(t) / (2 * PI) * one) % one
        off = min(off, one - off)
        assert off <= Fraction(1, 2) + Fraction(1, 2 ** 30), (t, float(off))


def test_turn_fraction_of_the_negative_is_the_negative(turn_fraction):
    for t in list(1e6 ** (-2.0 * np.arange(64) / 128)) + [7.5, 2.5e3, 1e-18]:
        assert (turn_fraction(float(t)) + turn_fraction(-float(t))) % 2 ** 64 == 0
