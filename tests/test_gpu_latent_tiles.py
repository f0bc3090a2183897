"""Long contexts, where a tile of rows that is stale, swapped or missing changes an output
by little: the norm of a row's error (attended_norm), and values that are 1 in the column of
their tile alone, which leave nothing to cancel."""
import numpy as np
import pytest
import torch

import position_invariant_kv_chunk_gb300 as K
from tests import attended_norm as N
from tests import latent_ref as L
from tests import paged_ref as R
from tests import test_gpu_latent as T
from tests import test_gpu_packed as P4
from tests.test_gpu_latent import BF, DEV, LORA, W, gen, i32, normal

pytestmark = pytest.mark.gpu


def one_column(n, tile, width):
    """[n, width]: row t is 1 in column t // tile (modulo the width)."""
    return (torch.arange(n, device=DEV)[:, None] // tile % width == torch.arange(width, device=DEV)).to(BF)


@pytest.mark.parametrize("Hq,P,lens", [(16, 64, [40000]), (32, 16, [9000, 1, 20000]), (33, 64, [9000, 4000]), (64, 128, [30001]),
                                       (100, 16, [9000, 0, 5003]), (128, 64, [40000]), (128, 48, [9000] * 4)])
def test_decode(Hq, P, lens):
    pool = T.Pool(Hq + P, sum(-(-x // P) for x in lens) + 1, P)
    table = pool.table(lens)
    q = normal(pool.g, len(lens), Hq, W)
    some = [0, Hq // 2, Hq - 1]
    slots = [R.slots_of(table[s].tolist(), P, n, pool.n) for s, n in enumerate(lens)]

    def call():
        pool.poison()
        out, lse = K.kamera_mla_attend_paged(pool.kv, LORA, q, P, table, i32(lens), max(lens))
        rows = [R.f64(pool.kv[torch.from_numpy(x).to(DEV)]) for x in slots]
        return out[:, some], lse[:, some], R.f64(q)[:, some], rows
    out, _, qh, rows = call()
    refs = [r for s in range(len(lens)) for r in N.rows(qh[s], rows[s], rows[s][:, :LORA], W ** -0.5)]
    N.near(out, refs, W, T.weight_error(Hq), (Hq, P))
    q[:, :, :LORA] = 0
    for x in slots:
        pool.kv[torch.from_numpy(x).to(DEV), :LORA] = one_column(len(x), 64, LORA)
    out, lse, qh, rows = call()
    refs = [r for s in range(len(lens)) for r in L.latent_rows(qh[s], rows[s], LORA, W ** -0.5)]
    L.near(out, lse, refs, W, T.weight_error(Hq), (Hq, P))


@pytest.mark.parametrize("seqs,H,nq,nk,causal", [(1, 2, 130, 9000, True), (1, 1, 3, 8191, True), (1, 3, 200, 2500, False),
                                                 (4, 40, 290, 1300, True), (2, 128, 257, 2000, True)])
def test_prefill(seqs, H, nq, nk, causal):
    g = gen(nk + H)
    qs, ks = T.starts([nq] * seqs), T.starts([nk] * seqs)
    q, kv, kr = normal(g, qs[-1], H, 192), normal(g, ks[-1], H, 256), normal(g, ks[-1], 64)
    pairs = sorted({(0, 0), (seqs - 1, H - 1), (seqs // 2, H // 2)})
    seen = range(0, nq, 9)

    def call():
        out, lse = K.kamera_mla_prefill_attend(q, kv, kr, i32(qs), i32(ks), nq, causal=causal)
        torch.cuda.synchronize()
        for s, h in pairs:
            a, b, c, d = qs[s], qs[s + 1], ks[s], ks[s + 1]
            k = np.concatenate([R.f64(kv[c:d, h, :128]), R.f64(kr[c:d])], axis=1)
            yield out[a:b, h], lse[a:b, h], R.f64(q[a:b, h]), k, R.f64(kv[c:d, h, 128:])
    for out, _, qh, k, v in call():
        refs = [N.rows(qh[i:i + 1], k[:m], v[:m], 192 ** -0.5)[0] for i in seen for m in [i + 1 + nk - nq if causal else nk]]
        N.near(out[list(seen)], refs, 192, 2.0 ** -8, (H, nk))
    q[:, :, :128] = 0
    for s in range(seqs):
        kv[ks[s]:ks[s + 1], :, 128:] = one_column(nk, 64, 128)[:, None]
    for out, lse, qh, k, v in call():
        L.near(out, lse, L.prefill_rows(qh, k, v, 192 ** -0.5, causal), 192, 2.0 ** -8, (H, nk))


@pytest.mark.parametrize("H,G,d,lens", [(4, 7, 128, [30000, 0, 12001]), (1, 1, 128, [40000]), (2, 12, 64, [21000, 5])])
def test_packed(H, G, d, lens):
    c = P4.Cache(H + G, lens, [9] * len(lens), H, d, 16)
    q = normal(c.g, len(lens), H * G, d)
    out, _ = K.kamera_attend_packed(*c.args(q))
    torch.cuda.synchronize()
    qf, tk, tv, refs = R.f64(q), R.f64(c.tk), R.f64(c.tv), []
    for s, n in enumerate(lens):
        at, ts = c.rows[s][0] * 16 + np.arange(n), c.tail_slots[s]
        for h in range(H):
            refs += N.rows(qf[s, h * G:h * G + G], np.concatenate([c.pk[at, h], tk[ts, h]]),
                           np.concatenate([c.pv[at, h], tv[ts, h]]), d ** -0.5)
    N.near(out, refs, d, P4.HALF, (H, G))


@pytest.mark.parametrize("H,G,d,n", [(2, 7, 128, 30000), (3, 1, 128, 9001), (2, 12, 64, 20000)])
def test_packed_one_column_a_tile(H, G, d, n):
    """A tile is 128 tokens; the last ones are the tail's."""
    P, g = 16, gen(n)
    pages, tail = n // P, n % P
    k = normal(g, pages * P, H, d)
    v = one_column(pages * P, 128, d)[:, None].expand(-1, H, -1).contiguous()
    packed = P4.packed_like(pages, H, P, d, fill=0xFF)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    K.kamera_pack_pages(k, v, P, torch.arange(pages, dtype=torch.int32, device=DEV), i32([P] * pages), packed, order)
    q, tk, tv = normal(g, 1, H * G, d), normal(g, P, H, d), torch.zeros(P, H, d, dtype=BF, device=DEV)
    out, lse = K.kamera_attend_packed(packed, q, P, order[None], i32([pages * P]), pages * P, tk, tv, i32([[0]]), i32([tail]), P)
    torch.cuda.synchronize()
    pk, pv = P4.pack_ref(k, v, P, pages)
    qf, refs = R.f64(q), []
    for h in range(H):
        kk = np.concatenate([pk[:, h], R.f64(tk)[:tail, h]])
        vv = np.concatenate([pv[:, h], R.f64(tv)[:tail, h]])
        o, l, m, x = R.attention(qf[0, h * G:h * G + G], kk, vv, d ** -0.5)
        refs += [(o[j], l[j], m[j], x[j], len(kk), np.abs(vv).sum(0)) for j in range(G)]
    L.near(out, lse, refs, d, P4.HALF, (H, G), P4.LEAST)
