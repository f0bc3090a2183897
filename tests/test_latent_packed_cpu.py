"""Latent attention over the paged pool and pages in 4 bits without a GPU: refusals,
struct layouts and workspace sizes.  No call here launches a kernel: every one returns
at its argument checks."""
import ctypes as C
import subprocess

import pytest
import torch

import position_invariant_kv_chunk_gb300 as K
from position_invariant_kv_chunk_gb300 import build as B

BF = torch.bfloat16
INVALID, MISALIGNED, UNSUPPORTED = 1, 2, 3
BASE = 1 << 30   # an address that no check dereferences
MB = 1 << 20
host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="host-only argument checks; run where no GPU exists")


def test_struct_layouts_match_header(tmp_path):
    structs = {"KameraPagedMlaKV": K._PagedMlaKV, "KameraMlaExpand": K._MlaExpand, "KameraMlaPrefill": K._MlaPrefill,
               "KameraPackedPool": K._PackedPool}
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


# ---------------------------------------------------------- absorbed decode --
def decode_args(**kw):
    v = dict(kv=BASE, num_slots=4096, slot_stride=576, kv_lora_rank=512, rope_dim=64, page_size=16, q=BASE + 64 * MB,
             out=BASE + 80 * MB, lse=BASE + 96 * MB, n_seqs=6, num_q_heads=16, scale=0.1, pages=BASE + 97 * MB,
             lens=BASE + 98 * MB, max_pages=64, max_len=1000, ws=BASE + 256 * MB, ws_bytes=1 << 34)
    assert set(kw) <= set(v)
    v.update(kw)
    return (K._PagedMlaKV(v["kv"], v["num_slots"], v["slot_stride"], v["kv_lora_rank"], v["rope_dim"], v["page_size"], 0),
            K._PagedQuery(v["q"], v["out"], v["lse"], v["n_seqs"], v["num_q_heads"], v["scale"], 0),
            K._PageTable(v["pages"], v["lens"], v["max_pages"], v["max_len"]), v["ws"], v["ws_bytes"])


@pytest.mark.parametrize("kw,status", [
    (dict(kv_lora_rank=256, slot_stride=576), UNSUPPORTED), (dict(rope_dim=32), UNSUPPORTED),
    (dict(num_q_heads=129), UNSUPPORTED), (dict(num_q_heads=0), INVALID), (dict(page_size=24), UNSUPPORTED),
    (dict(page_size=0), INVALID), (dict(n_seqs=65536), UNSUPPORTED), (dict(n_seqs=-1), INVALID),
    (dict(max_len=1025), INVALID), (dict(max_len=-1), INVALID), (dict(max_pages=-1), INVALID),
    (dict(num_slots=1 << 31), UNSUPPORTED), (dict(scale=float("nan")), INVALID), (dict(slot_stride=568), INVALID),
    (dict(slot_stride=580), MISALIGNED), (dict(kv=BASE + 8), MISALIGNED), (dict(kv=0), INVALID), (dict(q=0), INVALID),
    (dict(out=0), INVALID), (dict(lens=0), INVALID), (dict(pages=0), INVALID), (dict(q=BASE + 64 * MB + 8), MISALIGNED),
    (dict(out=BASE + 80 * MB + 2), MISALIGNED), (dict(lse=BASE + 96 * MB + 1), MISALIGNED),
    (dict(pages=BASE + 97 * MB + 2), MISALIGNED), (dict(ws=0), INVALID), (dict(ws_bytes=64), INVALID),
    (dict(ws=BASE + 256 * MB + 4), MISALIGNED), (dict(ws=BASE), INVALID), (dict(out=BASE), INVALID),
    (dict(out=BASE + 64 * MB), INVALID), (dict(lse=BASE + 80 * MB), INVALID), (dict(lse=BASE + 98 * MB), INVALID),
])
def test_decode_refusals(kw, status):
    kv, q, t, ws, n = decode_args(**kw)
    assert K.load_library().kamera_mla_attend_paged(C.byref(kv), C.byref(q), C.byref(t), ws, n, None, None) == status, kw


def test_decode_of_nothing_is_ok():
    kv, q, t, ws, n = decode_args(n_seqs=0)
    lib = K.load_library()
    assert lib.kamera_mla_attend_paged(C.byref(kv), C.byref(q), C.byref(t), None, 0, None, None) == 0
    assert lib.kamera_mla_attend_paged_workspace_bytes(C.byref(kv), C.byref(q), C.byref(t)) == 0


# --------------------------------------------------------------- expansion --
@pytest.mark.parametrize("kw,status", [
    (dict(kv_lora_rank=256), UNSUPPORTED), (dict(rope_dim=128, slot_stride=640), UNSUPPORTED),
    (dict(head_width=320), UNSUPPORTED), (dict(num_heads=129), UNSUPPORTED), (dict(num_heads=0), INVALID),
    (dict(n_tokens=-1), INVALID), (dict(weight=0), INVALID), (dict(slots=0), INVALID), (dict(kv_out=0), INVALID),
    (dict(k_rope_out=0), INVALID), (dict(kv=0), INVALID), (dict(weight=BASE + 64 * MB + 8), MISALIGNED),
    (dict(slots=BASE + 100 * MB + 4), MISALIGNED), (dict(kv_out=BASE + 128 * MB + 8), MISALIGNED),
    (dict(slot_stride=568), INVALID), (dict(slot_stride=580), MISALIGNED), (dict(kv_out=BASE), INVALID),
    (dict(kv_out=BASE + 64 * MB), INVALID), (dict(k_rope_out=BASE + 128 * MB), INVALID), (dict(k_rope_out=BASE), INVALID),
    (dict(n_tokens=0), 0),
])
def test_expand_refusals(kw, status):
    v = dict(kv=BASE, num_slots=4096, slot_stride=576, kv_lora_rank=512, rope_dim=64, weight=BASE + 64 * MB,
             slots=BASE + 100 * MB, kv_out=BASE + 128 * MB, k_rope_out=BASE + 512 * MB, n_tokens=100, num_heads=16,
             head_width=256)
    v.update(kw)
    kv = K._PagedMlaKV(v["kv"], v["num_slots"], v["slot_stride"], v["kv_lora_rank"], v["rope_dim"], 0, 0)
    x = K._MlaExpand(v["weight"], v["slots"], v["kv_out"], v["k_rope_out"], v["n_tokens"], v["num_heads"], v["head_width"],
                     0)
    assert K.load_library().kamera_mla_expand(C.byref(kv), C.byref(x), None, None) == status, kw


# ----------------------------------------------------------------- prefill --
@pytest.mark.parametrize("kw,status", [
    (dict(nope_dim=64), UNSUPPORTED), (dict(rope_dim=32), UNSUPPORTED), (dict(v_dim=64), UNSUPPORTED),
    (dict(num_heads=129), UNSUPPORTED), (dict(num_heads=0), INVALID), (dict(n_q=-1), INVALID), (dict(max_q=-1), INVALID),
    (dict(n_kv=(1 << 30) + 1), UNSUPPORTED), (dict(scale=float("nan")), INVALID), (dict(q=0), INVALID),
    (dict(kv=0), INVALID), (dict(k_rope=0), INVALID), (dict(out=0), INVALID), (dict(q_start=0), INVALID),
    (dict(kv_start=0), INVALID), (dict(q_stride=188), INVALID), (dict(q_stride=16 * 192 + 4), MISALIGNED),
    (dict(q_head_stride=184), INVALID), (dict(kv_stride=16 * 256 - 8), INVALID), (dict(kv_stride=16 * 256 + 4), MISALIGNED),
    (dict(k_rope_stride=56), INVALID), (dict(k_rope=BASE + 65 * MB + 8), MISALIGNED), (dict(out=BASE + 8), MISALIGNED),
    (dict(lse=BASE + 97 * MB + 2), MISALIGNED), (dict(q_start=BASE + 98 * MB + 1), MISALIGNED), (dict(out=BASE), INVALID),
    (dict(out=BASE + 32 * MB), INVALID), (dict(lse=BASE + 80 * MB), INVALID), (dict(n_seqs=0), 0), (dict(n_q=0), 0),
    (dict(max_q=0), 0), (dict(max_q=1 << 30, n_seqs=1 << 20), UNSUPPORTED),
])
def test_prefill_refusals(kw, status):
    v = dict(q=BASE, kv=BASE + 32 * MB, k_rope=BASE + 65 * MB, out=BASE + 80 * MB, lse=BASE + 97 * MB,
             q_start=BASE + 98 * MB, kv_start=BASE + 99 * MB, q_stride=16 * 192, q_head_stride=192, kv_stride=16 * 256,
             k_rope_stride=64, n_q=100, n_kv=300, n_seqs=2, num_heads=16, nope_dim=128, rope_dim=64, v_dim=128, max_q=60,
             causal=1, scale=0.1)
    v.update(kw)
    x = K._MlaPrefill(*[v[f] for f, _ in K._MlaPrefill._fields_])
    assert K.load_library().kamera_mla_prefill_attend(C.byref(x), None, None) == status, kw


# ------------------------------------------------------------------- pages --
PACK = dict(num_layers=2, num_kv_heads=4, head_dim=128, k=BASE, v=BASE + 64 * MB, num_slots=4096, layer_stride=4096 * 512,
            slot_stride=512, layer=1, data=BASE + 128 * MB, num_pages=256, page_size=16, k_unit=1.0, v_unit=0.25,
            kv_pages=BASE + 256 * MB, packed_pages=BASE + 257 * MB, tokens=BASE + 258 * MB, n=10)


@pytest.mark.parametrize("kw,status", [
    (dict(layer=2), INVALID), (dict(layer=-1), INVALID), (dict(n=-1), INVALID), (dict(head_dim=96), UNSUPPORTED),
    (dict(page_size=24), UNSUPPORTED), (dict(page_size=0), INVALID), (dict(k_unit=3.0), INVALID),
    (dict(v_unit=0.0), INVALID), (dict(k_unit=-1.0), INVALID), (dict(k_unit=float("inf")), INVALID),
    (dict(v_unit=float("nan")), INVALID), (dict(v_unit=2.0 ** 65), INVALID), (dict(num_pages=-1), INVALID),
    (dict(num_slots=1 << 31, layer_stride=1 << 41), UNSUPPORTED), (dict(k=0), INVALID), (dict(data=0), INVALID),
    (dict(kv_pages=0), INVALID), (dict(packed_pages=0), INVALID), (dict(tokens=0), INVALID),
    (dict(slot_stride=504), INVALID), (dict(slot_stride=516), MISALIGNED), (dict(data=BASE + 128 * MB + 8), MISALIGNED),
    (dict(tokens=BASE + 258 * MB + 2), MISALIGNED), (dict(data=BASE), INVALID), (dict(v=BASE), INVALID), (dict(n=0), 0),
])
@pytest.mark.parametrize("pack", [True, False])
def test_pack_refusals(kw, status, pack):
    assert pack_status(pack, **kw) == status, kw


def pack_status(pack, **kw):
    v = {**PACK, **kw}
    pool = K._GqaPool(*[v.get(f, 0) for f, _ in K._GqaPool._fields_])
    packed = K._PackedPool(v["data"], v["num_pages"], v["num_kv_heads"], v["head_dim"], v["page_size"], 0, v["k_unit"],
                           v["v_unit"])
    lib = K.load_library()
    call = lib.kamera_pack_pages if pack else lib.kamera_unpack_pages
    return call(C.byref(pool), v["layer"], C.byref(packed), v["kv_pages"], v["packed_pages"], v["tokens"], v["n"], None, None)


def test_pack_refuses_lists_in_what_it_writes():
    assert pack_status(True, tokens=BASE + 128 * MB) == INVALID
    assert pack_status(False, kv_pages=BASE + 64) == INVALID


def packed_args(**kw):
    v = dict(data=BASE, num_pages=1024, num_kv_heads=2, head_dim=128, page_size=16, k_unit=1.0, v_unit=1.0,
             q=BASE + 64 * MB, out=BASE + 65 * MB, lse=BASE + 66 * MB, n_seqs=6, num_q_heads=14, scale=0.1,
             pages=BASE + 67 * MB, lens=BASE + 68 * MB, max_pages=64, max_len=1000, k=BASE + 128 * MB, v=BASE + 160 * MB,
             num_slots=4096, slot_stride=256, tail_heads=2, tail_dim=128, tail_page=32, tail_pages=BASE + 69 * MB,
             tail_lens=BASE + 70 * MB, tail_max_pages=2, max_tail=64, ws=BASE + 256 * MB, ws_bytes=1 << 34)
    assert set(kw) <= set(v)
    v.update(kw)
    return (K._PackedPool(v["data"], v["num_pages"], v["num_kv_heads"], v["head_dim"], v["page_size"], 0, v["k_unit"],
                          v["v_unit"]),
            K._PagedQuery(v["q"], v["out"], v["lse"], v["n_seqs"], v["num_q_heads"], v["scale"], 0),
            K._PageTable(v["pages"], v["lens"], v["max_pages"], v["max_len"]),
            K._PagedKV(v["k"], v["v"], v["num_slots"], v["slot_stride"], v["tail_heads"], v["tail_dim"], v["tail_page"], 0),
            K._PageTable(v["tail_pages"], v["tail_lens"], v["tail_max_pages"], v["max_tail"]), v["ws"], v["ws_bytes"])


@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=96, tail_dim=96), UNSUPPORTED), (dict(num_q_heads=34), UNSUPPORTED), (dict(num_q_heads=13), INVALID),
    (dict(page_size=24), UNSUPPORTED), (dict(k_unit=0.3), INVALID), (dict(n_seqs=-1), INVALID),
    (dict(n_seqs=40000), UNSUPPORTED), (dict(max_len=1025), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(tail_heads=4, num_q_heads=16, slot_stride=512), INVALID), (dict(tail_dim=64), INVALID),
    (dict(max_tail=65), INVALID), (dict(tail_page=24, max_tail=40), UNSUPPORTED), (dict(slot_stride=248), INVALID),
    (dict(slot_stride=260), MISALIGNED), (dict(data=0), INVALID), (dict(data=BASE + 8), MISALIGNED), (dict(q=0), INVALID),
    (dict(q=BASE + 64 * MB + 2), MISALIGNED), (dict(pages=0), INVALID), (dict(lens=0), INVALID), (dict(tail_lens=0), INVALID),
    (dict(tail_pages=BASE + 69 * MB + 1), MISALIGNED), (dict(ws=0), INVALID), (dict(ws_bytes=100), INVALID),
    (dict(ws=BASE + 256 * MB + 8), MISALIGNED), (dict(ws=BASE), INVALID), (dict(out=BASE), INVALID),
    (dict(out=BASE + 128 * MB), INVALID), (dict(out=BASE + 64 * MB), INVALID), (dict(lse=BASE + 65 * MB), INVALID),
])
def test_packed_refusals(kw, status):
    pool, q, t, kv, tail, ws, n = packed_args(**kw)
    call = K.load_library().kamera_attend_packed
    assert call(C.byref(pool), C.byref(q), C.byref(t), C.byref(kv), C.byref(tail), ws, n, None, None) == status, kw


def test_packed_tail_goes_together_and_nothing_is_ok():
    lib = K.load_library()
    pool, q, t, kv, tail, ws, n = packed_args()
    assert lib.kamera_attend_packed(C.byref(pool), C.byref(q), C.byref(t), C.byref(kv), None, ws, n, None, None) == INVALID
    assert lib.kamera_attend_packed(C.byref(pool), C.byref(q), C.byref(t), None, C.byref(tail), ws, n, None, None) == INVALID
    pool, q, t, kv, tail, ws, n = packed_args(n_seqs=0)
    assert lib.kamera_attend_packed(C.byref(pool), C.byref(q), C.byref(t), C.byref(kv), C.byref(tail), None, 0, None,
                                    None) == 0
    assert lib.kamera_attend_packed_workspace_bytes(C.byref(pool), C.byref(q), C.byref(t), C.byref(kv), C.byref(tail)) == 0


def test_workspace_sizes():
    pool, q = torch.zeros(640, 576, dtype=BF), torch.zeros(3, 16, 576, dtype=BF)
    assert K.kamera_mla_attend_paged_workspace_bytes(pool, 512, q, 16, 600) > 0
    assert K.kamera_mla_attend_paged_workspace_bytes(pool, 512, q[:0], 16, 600) == 0
    assert K.kamera_mla_attend_paged_workspace_bytes(pool, 500, q, 16, 600) == 0          # it would refuse the call
    packed, q = torch.zeros(40, 2, 16 * 72, dtype=torch.uint8), torch.zeros(3, 8, 64, dtype=BF)
    a = K.kamera_attend_packed_workspace_bytes(packed, q, 16, 600)
    b = K.kamera_attend_packed_workspace_bytes(packed, q, 16, 600, 40)
    assert b > a > 0 and K.kamera_attend_packed_workspace_bytes(packed, q, 16, 0) == 0
    with pytest.raises(ValueError):
        K.kamera_attend_packed_workspace_bytes(packed, q, 0, 600)


# ------------------------------------------------------------- the binding --
@host_only
def test_binding_refusals():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    pool, q = torch.zeros(64, 576, dtype=BF), torch.zeros(2, 4, 576, dtype=BF)
    decode = lambda **k: K.kamera_mla_attend_paged(**{**dict(pool=pool, kv_lora=512, q=q, page_size=16, pages=i32(2, 4),
                                                             lens=i32(2), max_len=64), **k})
    for bad in (dict(q=q[:, :, :500]), dict(pages=i32(3, 4)), dict(lens=i32(3)), dict(out=torch.zeros(2, 4, 576, dtype=BF)),
                dict(lse=torch.zeros(2, 4, dtype=torch.float64)), dict(pages=None), dict(max_len=1 << 40),
                dict(pool=pool.t())):
        with pytest.raises(ValueError):
            decode(**bad)
    for bad in (dict(pool=pool.float()), dict(pages=3), dict(page_size="x")):
        with pytest.raises(TypeError):
            decode(**bad)
    w, slots = torch.zeros(3, 256, 512, dtype=BF), torch.zeros(5, dtype=torch.int64)
    expand = lambda **k: K.kamera_mla_expand(**{**dict(pool=pool, kv_lora=512, weight=w, slots=slots), **k})
    for bad in (dict(weight=w.transpose(0, 1)), dict(weight=w[0]), dict(slots=slots.int()),
                dict(kv=torch.zeros(5, 3, 255, dtype=BF)), dict(k_rope=torch.zeros(5, 32, dtype=BF))):
        with pytest.raises(ValueError):
            expand(**bad)
    pf = dict(q=torch.zeros(7, 2, 192, dtype=BF), kv=torch.zeros(9, 2, 256, dtype=BF), k_rope=torch.zeros(9, 64, dtype=BF),
              q_start=i32(3), kv_start=i32(3), max_q=7)
    for bad in (dict(kv=pf["kv"][:, :1]), dict(k_rope=pf["k_rope"][:5]), dict(q_start=i32(4)), dict(kv_start=i32(3).long()),
                dict(out=torch.zeros(7, 2, 192, dtype=BF)), dict(q=pf["q"][:, :, ::2]), dict(max_q=1 << 33)):
        with pytest.raises(ValueError):
            K.kamera_mla_prefill_attend(**{**pf, **bad})
    pk, packed = torch.zeros(64, 2, 64, dtype=BF), torch.zeros(4, 2, 16 * 72, dtype=torch.uint8)
    pack = dict(pool_k=pk, pool_v=pk.clone(), page_size=16, src_pages=i32(3), page_tokens=i32(3), packed=packed,
                dst_pages=i32(3))
    for bad in (dict(packed=packed[:, :, :-1]), dict(packed=packed.short()), dict(page_tokens=i32(2)), dict(page_size=0),
                dict(pool_v=pk.float())):
        with pytest.raises(ValueError):
            K.kamera_pack_pages(**{**pack, **bad})
    with pytest.raises(TypeError):
        K.kamera_pack_pages(**{**pack, "k_unit": "one"})
    at = dict(packed=packed, q=torch.zeros(2, 8, 64, dtype=BF), page_size=16, pages=i32(2, 4), lens=i32(2), max_len=64)
    for bad in (dict(pool_k=pk), dict(pool_k=pk, pool_v=pk, tail_pages=i32(2, 1), tail_lens=i32(3), max_tail=16),
                dict(q=torch.zeros(2, 8, 128, dtype=BF)), dict(lens=None), dict(packed=packed[:, 0])):
        with pytest.raises(ValueError):
            K.kamera_attend_packed(**{**at, **bad})
