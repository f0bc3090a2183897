"""The bound of a wait that counts SM cycles.  Runs without a GPU."""
import ctypes as C
import subprocess

import pytest

from position_invariant_kv_chunk_gb300 import build as B


@pytest.fixture(scope="module")
def wait_cycles(tmp_path_factory):
    d = tmp_path_factory.mktemp("wait")
    (d / "t.cpp").write_text('#include "kamera_hostcheck.h"\n'
                             'extern "C" unsigned long long cycles(unsigned long long ns) { return kamera::wait_cycles(kamera::half_wait(ns)); }\n')
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-I", B.INCLUDE, "-I", B.CSRC, str(d / "t.cpp"),
                    "-o", str(d / "t.so")], check=True)
    f = C.CDLL(str(d / "t.so")).cycles
    f.restype, f.argtypes = C.c_ulonglong, [C.c_ulonglong]
    return f


def test_cycles_last_the_bound_at_the_highest_clock_and_never_wrap(wait_cycles):
    """2070 MHz; the integer division loses a cycle, which the 1000 cover."""
    last = 0
    for ns in [0, 1, 7, 1000, 10 ** 6, 10 ** 9, 3 * 10 ** 9] + [2 ** e + d for e in range(40, 64) for d in (-1, 0, 1)] + [2 ** 64 - 1]:
        got = wait_cycles(ns)
        assert got >= 2.07 * min(ns, 2 ** 62) and got >= 1000 and got >= last, ns
        last = got
    assert wait_cycles(2 ** 63) > 2 ** 63
