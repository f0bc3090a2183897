"""Calls of latent attention and of the packed pages at the edges of what they take."""
import numpy as np
import pytest
import torch

import position_invariant_kv_chunk_gb300 as K
from tests import latent_ref as L
from tests import paged_ref as R
from tests import test_gpu_latent as T
from tests import test_gpu_packed as P4
from tests.test_gpu_latent import DESCRIPTOR, DEV, LEN, gen, i32, normal

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("qs,ks,bit", [([0, 20, 60], [0, 30, 80], LEN), ([0, 0, 60], [0, 30, 80], LEN),
                                       ([0, 0, 0], [0, 30, 80], 0), ([0, 61, 61], [0, 30, 80], DESCRIPTOR),
                                       ([0, 0, 5], [0, 81, 80], DESCRIPTOR), ([0, 0, 5], [-1, 30, 80], DESCRIPTOR | LEN)])
def test_prefill_with_a_bound_of_no_queries(qs, ks, bit):
    """A sequence with more queries than max_q is reported where max_q is 0 too."""
    g = gen(5)
    q, kv, kr = normal(g, 60, 2, 192), normal(g, 80, 2, 256), normal(g, 80, 64)
    out, lse, err = torch.full((60, 2, 128), 5.0, dtype=BF, device=DEV), torch.full((60, 2), 5.0, device=DEV), i32([0])
    K.kamera_mla_prefill_attend(q, kv, kr, i32(qs), i32(ks), 0, out=out, lse=lse, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == bit and bool((out == 5).all()) and bool((lse == 5).all())


@pytest.mark.parametrize("H,G,d", [(2, 7, 128), (1, 12, 64)])
def test_packed_attention_with_a_bound_of_no_tokens(H, G, d):
    """Lengths behind a bound of 0 are reported, in either part (max_tail is 0 where a call
    does not give it), and their tokens left out; lengths of 0 are fine, and so are none."""
    c = P4.Cache(41, [130, 0, 16], [5, 0, 20], H, d, 16)
    q = normal(c.g, 3, H * G, d)
    packed, _, P, table, lens, top, tk, tv, tt, tl, most, TP = c.args(q)
    zero, err = i32([0, 0, 0]), i32([0])

    def call(*part, **tail):
        err.zero_()
        out = K.kamera_attend_packed(packed, q, P, *part, **tail, tail_page_size=TP, err=err)
        torch.cuda.synchronize()
        return out, int(err.item())
    tail = dict(pool_k=tk, pool_v=tv, tail_pages=tt, tail_lens=tl, max_tail=most)
    no_tail = {**tail, "tail_lens": zero, "max_tail": 0}
    alone, bits = call(table, lens, top)
    assert bits == 0
    for part, kw, ref, bit in (((table, lens, top), {**tail, "max_tail": 0}, alone, LEN), ((table, lens, top), no_tail, alone, 0),
                               ((table, lens, 0), {}, None, LEN), ((table, zero, 0), {}, None, 0), ((None, None, 0), {}, None, 0),
                               ((table, lens, 0), no_tail, None, LEN), ((None, None, 0), {**tail, "max_tail": 0}, None, LEN)):
        (out, lse), bits = call(*part, **kw)
        assert bits == bit, (part[2], kw.get("max_tail"))
        if ref is None:
            assert not bool(out.any()) and bool((lse == -float("inf")).all())
        else:
            assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    (out, lse), bits = call(table, lens, 0, **tail)                    # the tails alone
    assert bits == LEN
    (want, wl), bits = call(None, None, 0, **tail)
    assert bits == 0 and torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("Hq,nope", [(16, 128), (40, 128), (4, 0)])
def test_decode_scaled_for_the_heads_before_the_absorption(Hq, nope):
    """nope_dim gives the scale of the expanded heads' keys, the one that prefill takes."""
    lens = [200, 0, 65]
    pool = T.Pool(Hq, 30, 16)
    table = pool.table(lens)
    q = normal(pool.g, 3, Hq, T.W)
    args = (pool.kv, T.LORA, q, 16, table, i32(lens), 200)
    scale = float(np.float32((nope + 64) ** -0.5))
    out, lse = K.kamera_mla_attend_paged(*args, nope_dim=nope)
    same, sl = K.kamera_mla_attend_paged(*args, scale=(nope + 64) ** -0.5)
    torch.cuda.synchronize()
    assert torch.equal(out, same) and torch.equal(lse, sl)
    L.near(out, lse, T.decode_refs(q, pool, table, lens, scale), T.W, T.weight_error(Hq), (Hq, nope))


@pytest.mark.parametrize("tokens,H", [(1, 128), (300, 128), (2000, 100), (700, 40)])
def test_expansion_of_many_heads(tokens, H):
    g = gen(tokens + H)
    pool, weight = normal(g, tokens + 9, T.W), normal(g, H, 256, T.LORA, std=0.05)
    slots = torch.randperm(tokens + 9, generator=g, device=DEV)[:tokens]
    err = i32([0])
    kv, kr = K.kamera_mla_expand(pool, T.LORA, weight, slots, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(kr, pool[slots][:, T.LORA:])
    T.expand_near(kv, pool, weight, slots.cpu().numpy())


@pytest.mark.parametrize("Hq", [16, 128])
def test_latent_rows_past_32_bits(Hq):
    """Rows whose place in the pool, in elements and in bytes, passes 32 bits."""
    P, W, lens = 16, T.W, [90, 200]
    n = 2 ** 32 // (P * W) + 40                                     # pages; 8.6 GB
    g = gen(Hq)
    pool = torch.empty(n * P, W, dtype=BF, device=DEV)
    pages = [n - 1 - i for i in range(10)] + [2 ** 31 // (P * W) + i for i in range(10)]
    rows = torch.tensor([p * P + t for p in pages for t in range(P)], device=DEV)
    pool[rows] = normal(g, len(rows), W)
    table = [pages[0::3] + [-1] * 6, pages[1::3] + pages[2::3]]
    table = i32([row[:13] for row in table])
    q, weight = normal(g, 2, Hq, W), normal(g, 3, 256, T.LORA, std=0.05)
    err = i32([0])
    out, lse = K.kamera_mla_attend_paged(pool, T.LORA, q, P, table, i32(lens), 200, err=err)
    kv, kr = K.kamera_mla_expand(pool, T.LORA, weight, rows, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    refs = []
    for s, m in enumerate(lens):
        at = torch.tensor([int(table[s, t // P]) * P + t % P for t in range(m)], device=DEV)
        refs += L.latent_rows(R.f64(q)[s], R.f64(pool[at]), T.LORA, W ** -0.5)
    L.near(out, lse, refs, W, T.weight_error(Hq), Hq)
    here = pool[rows]
    assert torch.equal(kr, here[:, T.LORA:])
    T.expand_near(kv, here, weight, np.arange(len(rows)))


def test_packed_pages_past_32_bits():
    """Pages of either pool behind 2^31 elements and 2^32 bytes, both ways and read by attention."""
    P, H, d, G = 16, 4, 128, 7
    n, m = 2 ** 32 // (P * H * P * 9) + 30, 2 ** 31 // (P * H * d) + 30     # packed pages (4.3 GB), bf16 pages (4.3 GB a pool)
    g = gen(8)
    packed = torch.empty(n, H, P * (d + d // 8), dtype=torch.uint8, device=DEV)
    k, v = torch.empty(m * P, H, d, dtype=BF, device=DEV), torch.empty(m * P, H, d, dtype=BF, device=DEV)
    src, dst, back = [m - 1 - i for i in range(8)], [n - 1 - 2 * i for i in range(8)], [m - 20 - i for i in range(8)]
    rows = lambda pages: torch.tensor([p * P + t for p in pages for t in range(P)], device=DEV)
    k[rows(src)], v[rows(src)] = normal(g, 8 * P, H, d), normal(g, 8 * P, H, d)
    err = i32([0])
    K.kamera_pack_pages(k, v, P, i32(src), i32([P] * 8), packed, i32(dst), err=err)
    K.kamera_unpack_pages(packed, P, i32(dst), i32([P] * 8), k, v, i32(back), err=err)
    q = normal(g, 1, H * G, d)
    out, lse = K.kamera_attend_packed(packed, q, P, i32([dst]), i32([120]), 120, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    pk, pv = P4.pack_ref(k[rows(src)], v[rows(src)], P, 8)
    assert np.array_equal(R.f64(k[rows(back)]), pk) and np.array_equal(R.f64(v[rows(back)]), pv)
    refs = []
    for h in range(H):
        o, l, mag, x = R.attention(R.f64(q)[0, h * G:h * G + G], pk[:120, h], pv[:120, h], d ** -0.5)
        refs += [(o[j], l[j], mag[j], x[j], 120, np.abs(pv[:120, h]).sum(0)) for j in range(G)]
    L.near(out, lse, refs, d, P4.HALF, "packed", P4.LEAST)


def test_expanded_rows_and_outputs_past_32_bits():
    """Expanded rows, queries and outputs behind 2^31 elements."""
    H, n = 128, 2 ** 31 // (128 * 256) + 500
    g = gen(11)
    pool, weight = normal(g, 400, T.W), normal(g, H, 256, T.LORA, std=0.05)
    slots = torch.arange(n, device=DEV) % 400
    err = i32([0])
    kv, kr = K.kamera_mla_expand(pool, T.LORA, weight, slots, err=err)
    one, _ = K.kamera_mla_expand(pool, T.LORA, weight, slots[:400], err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for a in (0, n // 2, n - 400):
        assert torch.equal(kv[a:a + 400], one[slots[a:a + 400]]) and torch.equal(kr[a:a + 400], pool[slots[a:a + 400]][:, T.LORA:])
    nq, nk = 2 ** 31 // (H * 128) + 300, 150
    q = torch.empty(nq, H, 192, dtype=BF, device=DEV)
    for a in range(0, nq, 20000):
        q[a:a + 20000] = normal(g, min(20000, nq - a), H, 192)
    start = [0, 7, nq]
    out, lse = K.kamera_mla_prefill_attend(q, kv, kr, i32(start), i32([n - 2 * nk, n - nk, n]), nq, causal=False, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for h in (0, H - 1):
        for s, some in ((0, [0, 6]), (1, [7, nq // 2, nq - 130, nq - 1])):
            rows = slice(n - (2 - s) * nk, n - (1 - s) * nk)
            k = np.concatenate([R.f64(kv[rows, h, :128]), R.f64(kr[rows])], axis=1)
            refs = L.prefill_rows(R.f64(q[some, h]), k, R.f64(kv[rows, h, 128:]), 192 ** -0.5, False)
            L.near(out[some, h], lse[some, h], refs, 192, 2.0 ** -8, (h, s))


@pytest.mark.parametrize("seqs,H,scale", [(1, 2, 0.0), (1, 2, -0.0), (4, 40, 0.0), (1, 2, 2.0 ** -149)])
def test_prefill_of_large_scores_without_a_scale(seqs, H, scale):
    """A scale of zero weighs every row that is seen alike, scores of up to 2^125 too."""
    g = gen(13)
    nq, nk = 150, 300
    qs, ks = T.starts([nq] * seqs), T.starts([nk] * seqs)
    q, kv, kr = normal(g, qs[-1], H, 192), normal(g, ks[-1], H, 256), normal(g, ks[-1], 64)
    q[:, :, 1:], q[:, :, 0] = 0, 2.0 ** 62
    kv[:, :, 0] = torch.linspace(-8, 8, ks[-1], device=DEV)[:, None].to(BF) * 2.0 ** 60
    out, lse = K.kamera_mla_prefill_attend(q, kv, kr, i32(qs), i32(ks), nq, scale=scale)
    torch.cuda.synchronize()
    refs, seen = T.prefill_refs(q[:nq], kv[:nk], kr[:nk], [0, nq], [0, nk], 0.0, True)
    L.near(out[:nq], lse[:nq], refs, 192, 2.0 ** -8, (seqs, H, scale))


@pytest.mark.parametrize("Hq", [16, 40, 128])
def test_decode_beside_nan(Hq):
    """A query head that is NaN leaves the other heads, a sequence whose rows are NaN the
    sequences beside it in a CTA's share."""
    lens = [70, 300, 5, 40, 1000]
    pool = T.Pool(Hq, 100, 16)
    table = pool.table(lens)
    q = normal(pool.g, 5, Hq, T.W)
    args = (pool.kv, T.LORA, q, 16, table, i32(lens), 1000)
    refs = T.decode_refs(q, pool, table, lens, T.W ** -0.5)
    good, gl = K.kamera_mla_attend_paged(*args)
    rows = torch.from_numpy(R.slots_of(table[1].tolist(), 16, 300, 100)).to(DEV)
    kept = pool.kv[rows].clone()
    pool.kv[rows] = float("nan")
    out, lse = K.kamera_mla_attend_paged(*args)
    torch.cuda.synchronize()
    rest = [0, 2, 3, 4]
    assert torch.equal(out[rest], good[rest]) and torch.equal(lse[rest], gl[rest])
    assert bool(out[1].isnan().all()) and bool(lse[1].isnan().all())
    pool.kv[rows] = kept
    q[:, 3], q[0, Hq - 1, 7] = float("nan"), float("inf")
    out, lse = K.kamera_mla_attend_paged(*args)
    torch.cuda.synchronize()
    bad = torch.zeros(5, Hq, dtype=torch.bool, device=DEV)
    bad[:, 3] = bad[0, Hq - 1] = True
    assert bool(out[bad].isnan().all()) and bool(lse[bad].isnan().all())
    fine = (~bad).flatten().nonzero()[:, 0].tolist()
    L.near(out.flatten(0, 1)[fine], lse.flatten()[fine], [refs[i] for i in fine], T.W, T.weight_error(Hq), Hq)


def test_packed_attention_beside_nan():
    c = P4.Cache(51, [300, 40, 1000], [9, 20, 3], 2, 128, 16)
    q = normal(c.g, 3, 14, 128)
    args = c.args(q)
    refs = c.refs(q, 128 ** -0.5)
    good, gl = K.kamera_attend_packed(*args)
    c.tk[torch.from_numpy(c.tail_slots[1][:1]).to(DEV)] = float("nan")
    out, lse = K.kamera_attend_packed(*args)
    torch.cuda.synchronize()
    assert torch.equal(out[[0, 2]], good[[0, 2]]) and torch.equal(lse[[0, 2]], gl[[0, 2]]) and bool(out[1].isnan().all())
    q[:, 3] = float("nan")
    out, lse = K.kamera_attend_packed(*args)
    torch.cuda.synchronize()
    assert bool(out[:, 3].isnan().all()) and bool(lse[:, 3].isnan().all())
    fine = [i for i in range(3 * 14) if i % 14 != 3 and i // 14 != 1]
    L.near(out.flatten(0, 1)[fine], lse.flatten()[fine], [refs[i] for i in fine], 128, P4.HALF, "heads", P4.LEAST)


def test_prefill_of_heads_outermost_and_expansion_in_a_graph():
    """Queries whose heads lie further apart than their tokens; the expansion captured with
    the prefill that reads it, replayed on other inputs."""
    g = gen(61)
    H, nq, nk = 3, 200, 333
    pool, weight = normal(g, 500, T.W), normal(g, H, 256, T.LORA, std=0.05)
    slots = torch.randperm(500, generator=g, device=DEV)[:nk].contiguous()
    q = normal(g, H, nq, 192).transpose(0, 1)
    starts = i32([0, nq]), i32([0, nk])

    def call():
        kv, kr = K.kamera_mla_expand(pool, T.LORA, weight, slots)
        return kv, kr, *K.kamera_mla_prefill_attend(q, kv, kr, *starts, nq)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv, kr, out, lse = call()
    for _ in range(2):
        pool.copy_(normal(g, 500, T.W))
        q.copy_(normal(g, nq, H, 192))
        slots.copy_(torch.randperm(500, generator=g, device=DEV)[:nk])
        graph.replay()
        torch.cuda.synchronize()
        want = call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((kv, kr, out, lse), want))
        T.expand_near(kv, pool, weight, slots.cpu().numpy())
        refs, _ = T.prefill_refs(q, kv, kr, [0, nq], [0, nk], 192 ** -0.5, True)
        L.near(out, lse, refs, 192, 2.0 ** -8, "graph")


def test_packing_one_page_to_two_places():
    P, H, d = 32, 2, 64
    g = gen(71)
    k, v = normal(g, 4 * P, H, d), normal(g, 4 * P, H, d)
    packed = P4.packed_like(5, H, P, d)
    K.kamera_pack_pages(k, v, P, i32([2, 2, 0, 2]), i32([P, P, P, 20]), packed, i32([4, 0, 1, 3]))
    torch.cuda.synchronize()
    assert torch.equal(packed[4], packed[0]) and not bool(packed[2].any())
    piece = 18 * d
    assert torch.equal(packed[3, :, :piece], packed[0, :, :piece])


def test_workspace_of_a_larger_call_again():
    """One workspace for calls one behind another: nothing of the larger one's states is read."""
    lens = [900, 20, 3000, 64, 0, 700]
    pool = T.Pool(81, 400, 16)
    table = pool.table(lens)
    pool.poison()
    q = normal(pool.g, 6, 16, T.W)
    ws = torch.empty(K.kamera_mla_attend_paged_workspace_bytes(pool.kv, T.LORA, q, 16, 3000), dtype=torch.uint8, device=DEV)
    calls = [(list(range(6)), 3000), ([5, 1], 700), ([2], 3000), ([4, 3], 64), ([0, 1, 4], 900)]
    alone = [K.kamera_mla_attend_paged(pool.kv, T.LORA, q[s], 16, table[s].contiguous(), i32([lens[i] for i in s]), m)
             for s, m in calls]
    again = [K.kamera_mla_attend_paged(pool.kv, T.LORA, q[s], 16, table[s].contiguous(), i32([lens[i] for i in s]), m,
                                       workspace=ws) for s, m in calls]
    torch.cuda.synchronize()
    for a, b in zip(alone, again):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
