"""Host code of the decode-step entry points.  Runs without a GPU."""
import ctypes as C
import subprocess
from fractions import Fraction

import numpy as np
import pytest

import position_invariant_kv_chunk_gb300 as K
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


# -------------------------------------------------------------------- build --
@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The build's outputs in an empty folder, the library's compilation left out."""
    monkeypatch.setattr(B, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(B, "LIB_PATH", str(tmp_path / "libkamera.so"))
    monkeypatch.setattr(B, "BINDING_PATH", str(tmp_path / "_kamera_binding.so"))
    monkeypatch.setattr(B, "_build_library", lambda *a: (tmp_path / "libkamera.so").write_text("library"))
    return tmp_path


@pytest.mark.parametrize("where", ["_compile_binding", "_link_binding", "_torch_version"])
def test_library_is_built_where_the_binding_cannot_be(elsewhere, monkeypatch, where):
    """No g++ or headers, no libraries to link, no torch: the library is there all the
    same, ctypes callers go on, and a call through the binding says what is wrong."""
    def fails(*a):
        raise (ImportError if where == "_torch_version" else RuntimeError)("no such thing here")
    if where == "_link_binding":
        monkeypatch.setattr(B, "_compile_binding", lambda: "x.o")
    if where == "_torch_version":   # an older binding lies there, for a torch that is gone
        (elsewhere / "_kamera_binding.so").write_text("older")
        (elsewhere / "_kamera_binding.so.torch").write_text("older")
    monkeypatch.setattr(B, where, fails)
    with pytest.warns(UserWarning, match="no such thing here"):
        assert B.build() == B.LIB_PATH
    assert (elsewhere / "libkamera.so").read_text() == "library"
    with pytest.raises((RuntimeError, ImportError), match="no such thing here"):
        B.build_binding()
    if where != "_torch_version":
        monkeypatch.setattr(K, "_FAST", None)
        monkeypatch.setattr(K, "load_library", lambda: None)
        with pytest.raises(RuntimeError, match="no such thing here"):
            K.kamera_summarize_pages(None, 16, None, None, None)


def test_binding_of_older_sources_is_not_kept(elsewhere, monkeypatch):
    (elsewhere / "_kamera_binding.so").write_text("older")

    def fails():
        raise RuntimeError("no compiler")
    monkeypatch.setattr(B, "_compile_binding", fails)
    with pytest.warns(UserWarning, match="no compiler"):
        B.build()
    assert not (elsewhere / "_kamera_binding.so").exists()


def test_failing_library_still_raises(elsewhere, monkeypatch):
    def fails(*a):
        raise RuntimeError("nvcc failed")
    monkeypatch.setattr(B, "_build_library", fails)
    monkeypatch.setattr(B, "_compile_binding", lambda: "x.o")
    with pytest.raises(RuntimeError, match="nvcc failed"):
        B.build()
