"""The decode-step entry points without a GPU: their refusals, struct layouts,
workspace sizes, and the 64-bit reference forms against independent identities.
No call here launches a kernel: every one returns at its argument checks."""
import ctypes as C
import subprocess

import numpy as np
import pytest
import torch

import position_invariant_kv_chunk_gb300 as K
from position_invariant_kv_chunk_gb300 import build as B
from tests import paged_ref as R

BF = torch.bfloat16
INVALID, MISALIGNED, UNSUPPORTED = 1, 2, 3
BASE = 1 << 30   # an address that no check dereferences
MB = 1 << 20


def test_struct_layouts_match_header(tmp_path):
    structs = {"KameraAppendRows": K._AppendRows, "KameraPagedKV": K._PagedKV, "KameraPagedQuery": K._PagedQuery,
               "KameraPageTable": K._PageTable, "KameraPrefixGroups": K._PrefixGroups,
               "KameraPageSelect": K._PageSelect, "KameraPrefillQuery": K._PrefillQuery}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "kamera.h"', 'int main(void){']
    for cname, py in structs.items():
        lines.append(f'printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    src = tmp_path / "probe.c"
    src.write_text("\n".join(lines + ["return 0;}"]))
    subprocess.run(["gcc", "-std=c11", "-I", B.INCLUDE, str(src), "-o", str(tmp_path / "probe")], check=True)
    out = subprocess.run([str(tmp_path / "probe")], capture_output=True, text=True, check=True).stdout
    got = {(s, f): int(v) for s, f, v in (ln.split() for ln in out.splitlines())}
    for cname, py in structs.items():
        assert got[(cname, "size")] == C.sizeof(py), cname
        for f, _ in py._fields_:
            assert got[(cname, f)] == getattr(py, f).offset, (cname, f)


# ------------------------------------------------------------------ append --
def append_args(**kw):
    """A valid call's structs with some fields replaced."""
    pool = dict(num_layers=2, num_kv_heads=2, head_dim=64, reserved=0, k=BASE, v=BASE + 64 * MB, num_slots=1024,
                layer_stride=1024 * 128, slot_stride=128)
    rows = dict(k=BASE + 128 * MB, v=BASE + 129 * MB, q=BASE + 130 * MB, q_out=BASE + 131 * MB, k_stride=128,
                v_stride=128, q_stride=512, q_head_stride=64, q_out_stride=512, q_out_head_stride=64,
                positions=BASE + 132 * MB, slots=BASE + 133 * MB, n_tokens=5, num_q_heads=8, layer=1, reserved=0)
    rope = dict(base=1e4, rot_dim=64, rot_offset=0, pairing=0)
    for f, v in kw.items():   # k and v name the rows' fields
        next(d for d in (rows, pool, rope) if f in d)[f] = v
    return (K._GqaPool(*[pool[f] for f, _ in K._GqaPool._fields_]),
            K._AppendRows(*[rows[f] for f, _ in K._AppendRows._fields_]),
            K._Rope(rope["base"], rope["rot_dim"], rope["rot_offset"], rope["pairing"], 0, None, None, None))


APPEND_REFUSED = [
    (dict(layer=2), INVALID), (dict(layer=-1), INVALID), (dict(n_tokens=-1), INVALID), (dict(slots=0), INVALID),
    (dict(positions=0), INVALID), (dict(q_out=0), INVALID), (dict(q=0), INVALID), (dict(num_q_heads=0), INVALID),
    (dict(k_stride=120), INVALID), (dict(k_stride=132), MISALIGNED), (dict(v_stride=0), INVALID),
    (dict(q_stride=448), INVALID), (dict(q_out_head_stride=56), INVALID), (dict(q_head_stride=68), INVALID), (dict(q_head_stride=68, q_stride=640), MISALIGNED),
    (dict(slots=BASE + 133 * MB + 4), MISALIGNED), (dict(positions=BASE + 4), MISALIGNED),
    (dict(q_out=BASE + 131 * MB + 8), MISALIGNED), (dict(head_dim=60), UNSUPPORTED), (dict(rot_dim=72), INVALID),
    (dict(rot_dim=40), UNSUPPORTED), (dict(rot_offset=4, rot_dim=16), UNSUPPORTED), (dict(pairing=2), UNSUPPORTED),
    (dict(q_out=BASE + 130 * MB + 128), INVALID),                      # shifted against q
    (dict(q_out=BASE + 128 * MB), INVALID),                            # over k
    (dict(q_out=BASE + 64 * MB), INVALID), (dict(k=BASE + 16), INVALID),   # the pool itself
    (dict(q_out=BASE + 130 * MB, q_out_stride=520), INVALID),          # in place with other strides
    (dict(base=0.0), INVALID), (dict(n_tokens=1, q_head_stride=68), MISALIGNED),
    (dict(n_tokens=1, k=BASE + 128 * MB + 8), MISALIGNED),
]


@pytest.mark.parametrize("kw,status", APPEND_REFUSED)
def test_append_refusals(kw, status):
    pool, rows, rope = append_args(**kw)
    assert K.load_library().kamera_append_kv(C.byref(pool), C.byref(rows), C.byref(rope), None, None) == status, kw


def test_append_of_nothing_is_ok():
    pool, rows, rope = append_args(n_tokens=0)
    assert K.load_library().kamera_append_kv(C.byref(pool), C.byref(rows), C.byref(rope), None, None) == 0
    mla = K._MlaPool(1, 512, 64, 0, BASE, 1024, 1024 * 576, 576)
    rows.layer = 0
    assert K.load_library().kamera_mla_append_kv(C.byref(mla), C.byref(rows), C.byref(rope), None, None) == 0
    bad = K._MlaPool(1, 500, 64, 0, BASE, 1024, 1024 * 576, 576)
    assert K.load_library().kamera_mla_append_kv(C.byref(bad), C.byref(rows), C.byref(rope), None, None) == UNSUPPORTED


# --------------------------------------------------------------- attention --
def shared_args(**kw):
    v = dict(k=BASE, v=BASE + 64 * MB, num_slots=4096, slot_stride=256, num_kv_heads=2, head_dim=128, page_size=16,
             q=BASE + 128 * MB, out=BASE + 129 * MB, lse=BASE + 130 * MB, n_seqs=6, num_q_heads=14, scale=0.1,
             group_start=BASE + 131 * MB, prefix_pages=BASE + 132 * MB, prefix_lens=BASE + 133 * MB, n_groups=2,
             prefix_max_pages=64, max_prefix=1000, max_group=4, pages=BASE + 134 * MB, lens=BASE + 135 * MB,
             max_pages=8, max_len=120, ws=BASE + 256 * MB, ws_bytes=1 << 34)
    assert set(kw) <= set(v), set(kw) - set(v)
    v.update(kw)
    kv = K._PagedKV(v["k"], v["v"], v["num_slots"], v["slot_stride"], v["num_kv_heads"], v["head_dim"],
                    v["page_size"], 0)
    q = K._PagedQuery(v["q"], v["out"], v["lse"], v["n_seqs"], v["num_q_heads"], v["scale"], 0)
    pre = K._PrefixGroups(v["group_start"], v["prefix_pages"], v["prefix_lens"], v["n_groups"], v["prefix_max_pages"],
                          v["max_prefix"], v["max_group"])
    own = K._PageTable(v["pages"], v["lens"], v["max_pages"], v["max_len"])
    return kv, q, pre, own, v["ws"], v["ws_bytes"]


SHARED_REFUSED = [
    (dict(head_dim=96, slot_stride=256), UNSUPPORTED), (dict(num_q_heads=34), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED),
    (dict(num_q_heads=13), INVALID), (dict(n_seqs=-1), INVALID), (dict(max_len=129), INVALID),
    (dict(max_prefix=1025), INVALID), (dict(max_group=7), INVALID), (dict(num_slots=1 << 31), UNSUPPORTED),
    (dict(scale=float("nan")), INVALID), (dict(slot_stride=248), INVALID), (dict(slot_stride=260), MISALIGNED),
    (dict(q=BASE + 128 * MB + 8), MISALIGNED), (dict(lse=BASE + 130 * MB + 2), MISALIGNED),
    (dict(pages=BASE + 134 * MB + 2), MISALIGNED), (dict(ws=0), INVALID), (dict(ws_bytes=100), INVALID),
    (dict(ws=BASE + 256 * MB + 8), MISALIGNED), (dict(ws=BASE), INVALID), (dict(ws=BASE + 134 * MB), INVALID),
    (dict(out=BASE + 128 * MB), INVALID), (dict(out=BASE + 64 * MB), INVALID), (dict(lse=BASE + 129 * MB), INVALID),
    (dict(pages=0), INVALID), (dict(group_start=0), INVALID), (dict(prefix_lens=0), INVALID), (dict(q=0), INVALID),
    (dict(n_seqs=40000), UNSUPPORTED), (dict(max_pages=-1), INVALID), (dict(n_groups=-1), INVALID),
    (dict(k=0), INVALID), (dict(out=BASE + 133 * MB), INVALID), (dict(max_group=0), INVALID),
]


@pytest.mark.parametrize("kw,status", SHARED_REFUSED)
def test_shared_attention_refusals(kw, status):
    kv, q, pre, own, ws, n = shared_args(**kw)
    assert K.load_library().kamera_attend_shared(C.byref(kv), C.byref(q), C.byref(pre), C.byref(own), ws, n, None,
                                                 None) == status, kw


def test_workspace_sizes_follow_the_plan():
    lib = K.load_library()

    def size(**kw):
        kv, q, pre, own, _, _ = shared_args(**kw)
        return lib.kamera_attend_shared_workspace_bytes(C.byref(kv), C.byref(q), C.byref(pre), C.byref(own))

    rows, state = 6 * 14, 4 * 128 + 8
    assert size() >= rows * 2 * state                        # a prefix state and an own state a row at least
    assert size(n_groups=0, n_seqs=1, max_group=1, max_pages=512, max_len=8192) > 0   # many splits: a merge
    assert size(n_groups=0, max_len=120) == 0                # a few splits: joined in a cluster, no partial state
    assert size(head_dim=96) == 0 and size(n_seqs=0) == 0
    assert size(max_prefix=1024, prefix_max_pages=1 << 16) < 1 << 26
    kv, q, _, own, _, _ = shared_args(max_pages=4096, max_len=65536)
    a = lib.kamera_attend_selected_workspace_bytes(C.byref(kv), C.byref(q), C.byref(own), 1024)
    b = lib.kamera_attend_selected_workspace_bytes(C.byref(kv), C.byref(q), C.byref(own), 4)
    assert a > 0 and b == 0


def test_selected_attention_refusals():
    lib = K.load_library()
    kv, q, _, own, ws, n = shared_args()
    call = lambda sel, k, kv=kv, q=q, own=own, w=ws: lib.kamera_attend_selected(
        C.byref(kv), C.byref(q), C.byref(own), sel, k, w, n, None, None)
    assert call(0, 4) == INVALID and call(BASE + 140 * MB, -1) == INVALID
    assert call(BASE + 140 * MB + 2, 4) == MISALIGNED
    assert call(BASE + 129 * MB, 4) == INVALID                        # over the output
    assert call(BASE + 140 * MB, 1 << 28) == UNSUPPORTED


def select_args(**kw):
    v = dict(q=BASE, summary=BASE + MB, selected=BASE + 64 * MB, num_pages=1000, n_seqs=3, num_q_heads=8,
             num_kv_heads=2, head_dim=64, page_size=16, n_select=10, n_first=1, n_last=1, pages=BASE + 65 * MB,
             lens=BASE + 66 * MB, max_pages=500, max_len=8000, ws=BASE + 70 * MB, ws_bytes=3 * 2 * 500 * 8)
    assert set(kw) <= set(v)
    v.update(kw)
    x = K._PageSelect(*[v[f] for f, _ in K._PageSelect._fields_])
    return x, K._PageTable(v["pages"], v["lens"], v["max_pages"], v["max_len"]), v["ws"], v["ws_bytes"]


SELECT_REFUSED = [
    (dict(n_first=6, n_last=5), INVALID), (dict(n_first=-1), INVALID), (dict(n_select=-1, n_first=0, n_last=0), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(page_size=20), UNSUPPORTED), (dict(num_q_heads=34), UNSUPPORTED),
    (dict(num_q_heads=7), INVALID), (dict(max_len=8001), INVALID), (dict(q=0), INVALID), (dict(summary=0), INVALID),
    (dict(lens=0), INVALID), (dict(pages=0), INVALID), (dict(selected=0), INVALID), (dict(ws=0), INVALID),
    (dict(ws_bytes=23999), INVALID), (dict(ws=BASE + 70 * MB + 8), MISALIGNED), (dict(q=BASE + 2), MISALIGNED),
    (dict(selected=BASE + 64 * MB + 2), MISALIGNED), (dict(selected=BASE + 65 * MB), INVALID),
    (dict(ws=BASE + 64 * MB), INVALID), (dict(max_len=(1 << 21) + 1, max_pages=1 << 18), UNSUPPORTED),
    (dict(n_seqs=40000), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", SELECT_REFUSED)
def test_selection_refusals(kw, status):
    x, t, ws, n = select_args(**kw)
    assert K.load_library().kamera_select_pages(C.byref(x), C.byref(t), ws, n, None, None) == status, kw


def test_selection_workspace_is_a_key_per_page():
    x, t, _, _ = select_args()
    assert K.load_library().kamera_select_pages_workspace_bytes(C.byref(x), C.byref(t)) == 3 * 2 * 500 * 8
    x, t, _, _ = select_args(head_dim=96)
    assert K.load_library().kamera_select_pages_workspace_bytes(C.byref(x), C.byref(t)) == 0
    for kw in (dict(n_seqs=0), dict(n_select=0, n_first=0, n_last=0)):
        x, t, ws, n = select_args(**kw)
        assert K.load_library().kamera_select_pages(C.byref(x), C.byref(t), ws, n, None, None) == 0


def test_summary_refusals():
    lib = K.load_library()
    kv = lambda **kw: K._PagedKV(*[{**dict(k=BASE, v=0, num_slots=256, slot_stride=128, num_kv_heads=2, head_dim=64,
                                           page_size=16, reserved=0), **kw}[f] for f, _ in K._PagedKV._fields_])
    call = lambda kv, n=3, ids=BASE + MB, tok=BASE + 2 * MB, out=BASE + 3 * MB: lib.kamera_summarize_pages(
        C.byref(kv), ids, tok, n, out, None, None)
    assert call(kv(), n=0) == 0 and call(kv(), n=-1) == INVALID
    assert call(kv(page_size=8)) == UNSUPPORTED and call(kv(head_dim=60)) == UNSUPPORTED
    assert call(kv(slot_stride=120)) == INVALID and call(kv(k=BASE + 8)) == MISALIGNED
    assert call(kv(), ids=0) == INVALID and call(kv(), out=0) == INVALID and call(kv(), out=BASE) == INVALID
    assert call(kv(), out=BASE + 3 * MB + 8) == MISALIGNED and call(kv(), tok=BASE + 1) == MISALIGNED


# -------------------------------------------------------------- the binding --
def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses_what_the_library_cannot_see():
    rope = K.Rope(1e4, 64)
    pk = z(1, 32, 2, 64)
    k = z(4, 2, 64)
    pos, slots = z(4, dtype=torch.int64), z(4, dtype=torch.int64)
    A = K.kamera_append_kv
    bad = [
        lambda: A(pk.float(), pk, k, k, rope, pos, slots), lambda: A(pk[0], pk[0], k, k, rope, pos, slots),
        lambda: A(pk, pk[:, :16], k, k, rope, pos, slots), lambda: A(pk, pk.clone(), k[:, :1], k, rope, pos, slots),
        lambda: A(pk, pk.clone(), k, k[:3], rope, pos, slots), lambda: A(pk, pk.clone(), k, k, rope, pos[:3], slots),
        lambda: A(pk, pk.clone(), k, k, rope, pos, slots.int()), lambda: A(pk, pk.clone(), k, k, rope, None, slots),
        lambda: A(pk, pk.clone(), k, k, rope, pos, slots, q=z(4, 8, 32)),
        lambda: A(pk, pk.clone(), k, k, rope, pos, slots, q_out=z(4, 8, 64)),
        lambda: A(pk, pk.clone(), k, k, rope, pos, slots, q=z(4, 8, 64), q_out=z(4, 8, 64).float()),
        lambda: A(pk, pk.clone(), k.transpose(0, 1).contiguous().transpose(0, 1), k, rope, pos, slots),
        lambda: K.kamera_mla_append_kv(z(1, 8, 576), 512, z(4, 512), z(4, 32), rope, pos, slots),
        lambda: K.kamera_mla_append_kv(z(8, 576), 512, z(4, 512), z(4, 64), rope, pos, slots),
    ]
    pool = z(64, 2, 64)
    q, i = z(3, 4, 64), lambda *s: z(*s, dtype=torch.int32)
    S = K.kamera_attend_shared
    bad += [
        lambda: S(pool, pool[:32], q, 16, None, None, None, i(3, 2), i(3), 0, 0, 20),
        lambda: S(pool, pool, q[:, :, :32], 16, None, None, None, i(3, 2), i(3), 0, 0, 20),
        lambda: S(pool, pool, q.float(), 16, None, None, None, i(3, 2), i(3), 0, 0, 20),
        lambda: S(pool, pool, q, 16, None, None, None, i(2, 2), i(3), 0, 0, 20),
        lambda: S(pool, pool, q, 16, None, None, None, i(3, 2).long(), i(3), 0, 0, 20),
        lambda: S(pool, pool, q, 16, None, None, None, None, None, 0, 0, 20),
        lambda: S(pool, pool, q, 16, i(2), None, i(1), i(3, 2), i(3), 3, 16, 20),
        lambda: S(pool, pool, q, 16, i(3), i(1, 1), i(1), i(3, 2), i(3), 3, 16, 20),
        lambda: S(pool, pool, q, 16, None, None, None, i(3, 2), i(3), 0, 0, 20, out=z(3, 4, 32)),
        lambda: S(pool, pool, q, 16, None, None, None, i(3, 2), i(3), 0, 0, 20, lse=z(3, 4)),
        lambda: K.kamera_attend_selected(pool, pool, q, 16, i(3, 2), i(3), i(3, 1, 2), 20),
        lambda: K.kamera_select_pages(q, z(4, 2, 2, 32), 16, i(3, 2), i(3), 20, 2),
        lambda: K.kamera_select_pages(q, z(4, 2, 1, 64), 16, i(3, 2), i(3), 20, 2),
        lambda: K.kamera_select_pages(q, z(4, 2, 2, 64), 16, i(3, 2), i(3), 20, 2, selected=i(3, 2, 3)),
        lambda: K.kamera_summarize_pages(pool, 16, i(2), i(3), z(4, 2, 2, 64)),
        lambda: K.kamera_summarize_pages(pool, 16, i(2), i(2), z(5, 2, 2, 64)),
    ]
    for n, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
            pytest.fail(f"call {n} was accepted")


def test_binding_takes_cuda_tensors_only(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    i = lambda *s: z(*s, dtype=torch.int32)
    pk, pool, q = z(1, 32, 2, 64), z(64, 2, 64), z(3, 4, 64)
    j = z(4, dtype=torch.int64)
    for call in (
        lambda: K.kamera_append_kv(pk, pk.clone(), z(4, 2, 64), z(4, 2, 64), K.Rope(1e4, 64), j, j),
        lambda: K.kamera_mla_append_kv(z(1, 8, 576), 512, z(4, 512), z(4, 64), K.Rope(1e4, 64), j, j),
        lambda: K.kamera_attend_shared(pool, pool, q, 16, None, None, None, i(3, 2), i(3), 0, 0, 20),
        lambda: K.kamera_summarize_pages(pool, 16, i(2), i(2), z(4, 2, 2, 64)),
        lambda: K.kamera_select_pages(q, z(4, 2, 2, 64), 16, i(3, 2), i(3), 20, 2),
        lambda: K.kamera_attend_selected(pool, pool, q, 16, i(3, 2), i(3), i(3, 2, 2), 20),
    ):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


# ----------------------------------------------------- the reference's pins --
def test_reference_rotation_composes():
    """R(p) R(r) = R(p + r), and q at p against k at r depends on p - r alone."""
    rng = np.random.default_rng(1)
    inv = 1e4 ** (-2.0 * np.arange(16) / 32)
    for il in (False, True):
        x = rng.normal(size=(3, 2, 40))
        p, r = np.array([5, 0, 77]), np.array([-3, 11, 2])
        twice = R.turned(R.turned(x, p, inv, 8, il), r, inv, 8, il)
        assert np.allclose(twice, R.turned(x, p + r, inv, 8, il), atol=1e-12)
        assert np.array_equal(twice[..., :8], x[..., :8])
        y = rng.normal(size=(3, 2, 40))
        a = (R.turned(x, p, inv, 8, il) * R.turned(y, r, inv, 8, il)).sum(-1)
        assert np.allclose(a, (R.turned(x, p - r, inv, 8, il) * y).sum(-1), atol=1e-12)


def test_reference_attention_merges():
    """Attention over two halves, merged by their log-sum-exps, is attention over both."""
    rng = np.random.default_rng(2)
    q, k, v = rng.normal(size=(3, 8)), rng.normal(size=(11, 8)), rng.normal(size=(11, 8))
    o, l, _, _ = R.attention(q, k, v, 0.3)
    o1, l1, _, _ = R.attention(q, k[:4], v[:4], 0.3)
    o2, l2, _, _ = R.attention(q, k[4:], v[4:], 0.3)
    w1, w2 = np.exp(l1 - l)[:, None], np.exp(l2 - l)[:, None]
    assert np.allclose(w1 + w2, 1) and np.allclose(o, w1 * o1 + w2 * o2)


def test_reference_score_bounds_every_key():
    """A page's score is at least the heads' summed scores of any of its keys, and is
    reached by a key at the right corner of the box."""
    rng = np.random.default_rng(3)
    q, keys = rng.normal(size=(5, 12)), rng.normal(size=(7, 16, 12))
    s = R.page_scores(q, keys.min(1), keys.max(1))
    assert np.all((keys @ q.T).sum(-1).max(1) <= s + 1e-12)
    one = R.page_scores(q[:1], keys.min(1), keys.max(1))
    corner = np.where(q[0] > 0, keys.max(1), keys.min(1))
    assert np.allclose(one, corner @ q[0])
    assert R.select(np.array([5.0, 1, 9, 9, 2, 0]), 4, 1, 1) == [0, 2, 3, 5]
    assert R.select(np.array([5.0, 1, 9]), 5, 1, 1) == [0, 1, 2, -1, -1]
    assert R.select(np.array([0.0, 1, 1, 1, 0]), 3, 1, 1) == [0, 1, 4]
