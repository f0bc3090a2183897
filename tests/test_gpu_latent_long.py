"""Latent rows and packed pages at lengths at which a CTA's share is many tiles: pages
outside the pool in the middle of it, tokens without a row, calls at once.  References
and tolerances as in test_gpu_latent and test_gpu_packed."""
import numpy as np
import pytest
import torch

import position_invariant_kv_chunk_gb300 as K
from tests import latent_ref as L
from tests import paged_ref as R
from tests import test_gpu_latent as T
from tests import test_gpu_packed as P4
from tests.test_gpu_latent import DEV, LORA, SLOT, W, gen, i32, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,P,lens", [(16, 64, [60000, 1, 24000]), (32, 32, [80000]), (100, 16, [30000, 0, 14003]),
                                       (128, 64, [40000])])
def test_decode_of_long_contexts_with_bad_pages(Hq, P, lens):
    """Page tables that name pages again and again, and now and then none of the pool."""
    rng = np.random.default_rng(Hq)
    g, n = gen(Hq), 90
    pool = normal(g, n * P + 5, W + 8)[:, :W]
    pool[n * P:] = float("nan")
    table = rng.integers(0, n, (len(lens), -(-max(lens) // P)))
    table[rng.random(table.shape) < 0.03] = -1
    table[rng.random(table.shape) < 0.02] = n
    q = normal(g, len(lens), Hq, W)
    err = i32([0])
    out, lse = K.kamera_mla_attend_paged(pool, LORA, q, P, i32(table.tolist()), i32(lens), max(lens), err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == SLOT
    rows, refs, qh = R.f64(pool), [], R.f64(q)
    some = [0, Hq // 2, Hq - 1]
    for s, m in enumerate(lens):
        slots = R.slots_of(table[s], P, m, n)
        refs += L.latent_rows(qh[s][some], rows[slots[slots >= 0]], LORA, W ** -0.5)
    L.near(out[:, some], lse[:, some], refs, W, T.weight_error(Hq), (Hq, P))


@pytest.mark.parametrize("tokens,H", [(45037, 1), (20000, 3), (40961, 2)])
def test_expansion_of_many_tiles_with_bad_slots(tokens, H):
    g = gen(tokens)
    pool, weight = normal(g, 700, W), normal(g, H, 256, LORA, std=0.05)
    slots = torch.randint(0, 700, (tokens,), generator=g, device=DEV)
    dice = torch.rand(tokens, generator=g, device=DEV)
    slots[dice < 0.02] = -1
    slots[dice > 0.99] = 700
    slots[-1] = 2 ** 50
    err = i32([0])
    kv, kr = K.kamera_mla_expand(pool, LORA, weight, slots, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == SLOT
    there = (slots >= 0) & (slots < 700)
    assert torch.equal(kr[there], pool[slots[there]][:, LORA:])
    assert not bool(kr[~there].any()) and not bool(kv[~there].any())
    # one slot's outputs are the same wherever it stands
    one, _ = K.kamera_mla_expand(pool, LORA, weight, torch.arange(700, device=DEV))
    T.expand_near(one, pool, weight, np.arange(700))
    assert torch.equal(kv[there], one[slots[there]])


@pytest.mark.parametrize("H,G,lens", [(32, 1, [5100]), (4, 7, [30000, 0, 12001]), (8, 12, [21000])])
def test_packed_attention_of_long_contexts_with_bad_pages(H, G, lens):
    rng = np.random.default_rng(H)
    c = P4.Cache(H, lens, [9] * len(lens), H, 128, 16)
    left_out = set()
    for s, m in enumerate(lens):
        for j in range(-(-m // 16)):
            if rng.random() < 0.03:
                c.table[s, j] = int(rng.choice([-1, c.n, 2 ** 31 - 1]))
                left_out.add((s, j))
    q = normal(c.g, len(lens), H * G, 128)
    err = i32([0])
    out, lse = K.kamera_attend_packed(*c.args(q), err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == SLOT
    L.near(out, lse, c.refs(q, 128 ** -0.5, left_out=left_out), 128, P4.HALF, (H, G), P4.LEAST)


@pytest.mark.parametrize("seqs,H,nq,nk", [(1, 2, 130, 2500), (1, 1, 3, 1700), (4, 40, 290, 1300)])
def test_prefill_behind_long_prefixes(seqs, H, nq, nk):
    g = gen(nk)
    qs, ks = T.starts([nq] * seqs), T.starts([nk] * seqs)
    q, kv, kr = normal(g, qs[-1], H, 192), normal(g, ks[-1], H, 256), normal(g, ks[-1], 64)
    out, lse = K.kamera_mla_prefill_attend(q, kv, kr, i32(qs), i32(ks), nq)
    torch.cuda.synchronize()
    for s, h in {(0, 0), (seqs - 1, H - 1)}:
        a, b, c, d = qs[s], qs[s + 1], ks[s], ks[s + 1]
        k = np.concatenate([R.f64(kv[c:d, h, :128]), R.f64(kr[c:d])], axis=1)
        refs = L.prefill_rows(R.f64(q[a:b, h]), k, R.f64(kv[c:d, h, 128:]), 192 ** -0.5, True)
        L.near(out[a:b, h], lse[a:b, h], refs, 192, 2.0 ** -8, (s, h))


def test_calls_at_once():
    """All of them on four streams at the same time, each with buffers of its own."""
    g = gen(3)
    lens = [3000, 17, 900]
    pool = T.Pool(9, 300, 16)
    table = pool.table(lens)
    pool.poison()
    q = [normal(g, 3, h, W) for h in (16, 128)]
    weight, slots = normal(g, 4, 256, LORA, std=0.05), torch.from_numpy(R.slots_of(table[0].tolist(), 16, 3000, 300)).to(DEV)
    qp = normal(g, 500, 4, 192)
    c = P4.Cache(5, [4000, 100], [30, 3], 4, 128, 16)
    qd = normal(c.g, 2, 28, 128)

    def calls(stream):
        a = K.kamera_mla_attend_paged(pool.kv, LORA, q[0], 16, table, i32(lens), 3000, stream=stream)
        b = K.kamera_attend_packed(*c.args(qd), stream=stream)
        kv, kr = K.kamera_mla_expand(pool.kv, LORA, weight, slots, stream=stream)
        d = K.kamera_mla_prefill_attend(qp, kv, kr, i32([0, 500]), i32([0, 3000]), 500, stream=stream)
        e = K.kamera_mla_attend_paged(pool.kv, LORA, q[1], 16, table, i32(lens), 3000, stream=stream)
        return [*a, *b, kv, kr, *d, *e]
    ref = calls(torch.cuda.current_stream())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(3):
        outs = []
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(calls(s))
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(x, y) for x, y in zip(o, ref))
