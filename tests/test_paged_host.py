"""Host code of the decode-step entry points.  Runs without a GPU."""
import ctypes as C
import subprocess
from fractions import Fraction

import numpy as np
import pytest
import torch

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


# -------------------------------------------------------------- the binding --
def one_head(*lead, d=64):
    """bf16 [*lead, 1, d] whose single head has a stride of its own, which no element takes."""
    n = int(np.prod(lead))
    rows = [int(np.prod(lead[i + 1:])) * d for i in range(len(lead))]
    return torch.zeros(n * d, dtype=torch.bfloat16).as_strided((*lead, 1, d), (*rows, 40, 1))


def test_binding_looks_at_no_stride_that_is_not_taken(monkeypatch):
    """Pools of one head, or of one layer, whose size-1 dimensions have strides of any
    kind: calls without tokens, which end behind the checks of the pool."""
    monkeypatch.setattr(torch.cuda, "is_available", lambda: False)
    bf, i32 = torch.bfloat16, lambda *s: torch.zeros(*s, dtype=torch.int32)
    none = torch.zeros(0, dtype=torch.int64)
    rope = K.Rope(1e4, 64)
    for pk in (one_head(2, 32), torch.zeros(32 * 64, dtype=bf).as_strided((1, 32, 1, 64), (3, 64, 7, 1))):
        pv = torch.zeros(pk.shape, dtype=bf)
        rows = torch.zeros(0, 1, 64, dtype=bf)
        assert K.kamera_append_kv(pk, pv, rows, rows, rope, none, none) is None
        assert K.kamera_append_kv(pv, pk, rows, rows, rope, none, none) is None
    pool = torch.zeros(32 * 576, dtype=bf).as_strided((1, 32, 576), (5, 576, 1))
    assert K.kamera_mla_append_kv(pool, 512, torch.zeros(0, 512, dtype=bf), torch.zeros(0, 64, dtype=bf),
                                  K.Rope(1e4, 64, 0, K.INTERLEAVED), none, none) is None
    pk, q = one_head(64), torch.zeros(0, 4, 64, dtype=bf)
    pv = torch.zeros(pk.shape, dtype=bf)
    out, lse = K.kamera_attend_shared(pk, pv, q, 16, None, None, None, i32(0, 2), i32(0), 0, 0, 20)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    K.kamera_attend_selected(pk, pv, q, 16, i32(0, 2), i32(0), i32(0, 1, 2), 20)
    K.kamera_summarize_pages(pk, 16, i32(0), i32(0), torch.zeros(4, 1, 2, 64, dtype=bf))
    wide = torch.zeros(64, 2, 80, dtype=bf)[:, :, :64]           # two heads that are not packed: refused as before
    with pytest.raises(ValueError, match="packed heads"):
        K.kamera_summarize_pages(wide, 16, i32(0), i32(0), torch.zeros(4, 2, 2, 64, dtype=bf))
    with pytest.raises(ValueError, match="share"):
        K.kamera_attend_shared(pk, torch.zeros(64, 1, 72, dtype=bf)[:, :, :64], q, 16, None, None, None, i32(0, 2),
                               i32(0), 0, 0, 20)


def test_workspace_sizes_from_python():
    """The sizes the C entry points give for the same call, from the call's tensors."""
    lib, z = K.load_library(), lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    pool, q, summary = z(640, 2, 64), z(3, 8, 64), z(40, 2, 2, 64)
    kv, query = K._PagedKV(None, None, 640, 128, 2, 64, 16, 0), K._PagedQuery(None, None, None, 3, 8, 0.5, 0)
    own = lambda n: K._PageTable(None, None, -(-n // 16), n)
    for groups, most, prefix, n in ((2, 2, 600, 50), (0, 0, 0, 50), (0, 0, 0, 100000), (1, 3, 30000, 0), (3, 1, 0, 17)):
        pre = K._PrefixGroups(None, None, None, groups, -(-prefix // 16), prefix, most)
        want = lib.kamera_attend_shared_workspace_bytes(C.byref(kv), C.byref(query), C.byref(pre), C.byref(own(n)))
        assert K.kamera_attend_shared_workspace_bytes(pool, q, 16, groups, most, prefix, n) == want
        assert (want > 0) == (prefix > 0 or n > 10000)
    for k, n in ((4, 600), (2000, 100000)):
        want = lib.kamera_attend_selected_workspace_bytes(C.byref(kv), C.byref(query), C.byref(own(n)), k)
        assert K.kamera_attend_selected_workspace_bytes(pool, q, 16, k, n) == want and (want > 0) == (k > 1000)
    assert K.kamera_select_pages_workspace_bytes(q, summary, 16, 601, 5) == 3 * 2 * 38 * 8
    assert K.kamera_select_pages_workspace_bytes(q, summary, 16, 601, 5, 3, 3) == 0      # more forced than taken
    assert K.kamera_attend_shared_workspace_bytes(pool, q, 24, 1, 3, 100, 50) == 0       # a page size it refuses
    for call in (lambda: K.kamera_attend_shared_workspace_bytes(pool, q[:, :, :32], 16, 1, 3, 100, 50),
                 lambda: K.kamera_attend_shared_workspace_bytes(pool, q, 0, 1, 3, 100, 50),
                 lambda: K.kamera_attend_shared_workspace_bytes(pool, q, 16, 1, 3, 2 ** 31, 50),
                 lambda: K.kamera_attend_selected_workspace_bytes(pool[0], q, 16, 4, 50),
                 lambda: K.kamera_select_pages_workspace_bytes(q, summary[0], 16, 50, 4)):
        with pytest.raises(ValueError):
            call()
