"""Latent attention over the paged MLA pool: absorbed decode, expansion of latent rows
and prefill over expanded rows, against their definitions in 64 bits.  Tolerances:
latent_ref.near; a weight enters the second product as a bf16 hi + lo pair (2^-16, up to
32 heads of a decode step) or rounded to bf16 (2^-8)."""
import numpy as np
import pytest
import torch

import position_invariant_kv_chunk_gb300 as K
from tests import latent_ref as L
from tests import paged_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
SLOT, DESCRIPTOR, LEN, TIMEOUT = 1, 4, 8, 32
W, LORA = 576, 512
BF = torch.bfloat16


def normal(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * std).to(BF)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


class Pool:
    """A latent pool of one layer and page tables drawn from it; poison() makes NaN of
    what no table names."""

    def __init__(self, seed, n_pages, P, pad=0, std=1.0, extra=0):
        self.g, self.P, self.n = gen(seed), P, n_pages
        wide = normal(self.g, n_pages * P + extra, W + pad, std=std)
        self.kv = wide[:, :W]
        self.order = torch.randperm(n_pages, generator=self.g, device=DEV).tolist()
        self.used = torch.zeros(len(wide), dtype=torch.bool, device=DEV)

    def table(self, lens, width=None):
        width = max(-(-max(lens, default=0) // self.P), 1) if width is None else width
        rows = []
        for n in lens:
            pages = [self.order.pop() for _ in range(-(-n // self.P))]
            for j, g in enumerate(pages):
                self.used[g * self.P:g * self.P + min(self.P, n - j * self.P)] = True
            rows.append(pages + [2 ** 31 - 1] * (width - len(pages)))
        return i32(rows)

    def poison(self):
        self.kv[~self.used] = float("nan")


def weight_error(Hq):
    return 2.0 ** -16 if Hq <= 32 else 2.0 ** -8


def decode_refs(q, pool, table, lens, scale):
    qh, refs = R.f64(q), []
    for s, n in enumerate(lens):
        slots = R.slots_of(table[s].tolist(), pool.P, n, pool.n)
        rows = R.f64(pool.kv[torch.from_numpy(slots[slots >= 0]).to(DEV)])
        refs += L.latent_rows(qh[s], rows, LORA, scale)
    return refs


# -------------------------------------------------------------------- decode --
@pytest.mark.parametrize("Hq,P,lens", [
    (16, 16, [0, 1, 15, 16, 17, 63, 64, 65, 200]), (1, 64, [64, 63, 0, 129]), (5, 48, [700, 3]), (16, 128, [1000]),
    (17, 16, [33, 0, 130]), (32, 32, [257, 64, 1]), (33, 16, [100, 0, 65]), (64, 64, [300, 1]), (65, 16, [17, 190]),
    (100, 48, [0, 97]), (128, 16, [130, 64, 0, 5]), (128, 128, [513]),
])
def test_decode_matches_definition(Hq, P, lens):
    pool = Pool(Hq + P, sum(-(-x // P) for x in lens) + 2, P, pad=8 * (Hq % 3), extra=7)
    table = pool.table(lens)
    pool.poison()
    q = normal(pool.g, len(lens), Hq, W)
    err = i32([0])
    out, lse = K.kamera_mla_attend_paged(pool.kv, LORA, q, P, table, i32(lens), max(lens), err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    L.near(out, lse, decode_refs(q, pool, table, lens, W ** -0.5), W, weight_error(Hq), (Hq, P))


@pytest.mark.parametrize("Hq", [16, 128])
def test_decode_of_many_short_and_of_one_long(Hq):
    """Ranges that hold many sequences, and a sequence that many ranges share."""
    rng = np.random.default_rng(Hq)
    for lens in ([int(x) for x in rng.integers(0, 40, 400)], [9000], [0] * 5, [1] * 3 + [4000] + [0, 2]):
        pool = Pool(len(lens), sum(-(-x // 16) for x in lens) + 1, 16)
        table = pool.table(lens)
        pool.poison()
        q = normal(pool.g, len(lens), Hq, W)
        out, lse = K.kamera_mla_attend_paged(pool.kv, LORA, q, 16, table, i32(lens), max(max(lens), 1))
        L.near(out, lse, decode_refs(q, pool, table, lens, W ** -0.5), W, weight_error(Hq), (Hq, len(lens)))


@pytest.mark.parametrize("Hq", [16, 32, 128])
@pytest.mark.parametrize("scale", [W ** -0.5, -0.05, 0.0, 3.0])
def test_decode_of_growing_scores_and_scales(Hq, scale):
    """Rows that grow along the sequence move the running maximum in every tile; a
    negative scale, none, and a sharp one."""
    lens = [500, 130]
    pool = Pool(3, 60, 16)
    table = pool.table(lens)
    for s, n in enumerate(lens):
        slots = torch.from_numpy(R.slots_of(table[s].tolist(), 16, n, 60)).to(DEV)
        pool.kv[slots] = (pool.kv[slots].float() * torch.linspace(0.1, 4, n, device=DEV)[:, None]).to(BF)
    pool.poison()
    q = normal(pool.g, 2, Hq, W)
    out, lse = K.kamera_mla_attend_paged(pool.kv, LORA, q, 16, table, i32(lens), 500, scale=scale)
    L.near(out, lse, decode_refs(q, pool, table, lens, np.float32(scale).astype(float)), W, weight_error(Hq), (Hq, scale))


def test_decode_reports_bad_pages_and_lengths():
    """Pages outside the pool are left out, sequences of impossible length read as empty."""
    for Hq in (16, 128):
        lens = [300, 90, 64, 16]
        pool = Pool(5, 60, 16)
        table = pool.table(lens)
        pool.poison()
        q = normal(pool.g, 4, Hq, W)
        table[0, 3], table[0, 4:8], table[1, 5], table[2, 0] = -1, 60, 2 ** 31 - 1, -2 ** 31
        table[3, 0] = 99
        err = i32([0])
        out, lse = K.kamera_mla_attend_paged(pool.kv, LORA, q, 16, table, i32(lens), 300, err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == SLOT
        L.near(out, lse, decode_refs(q, pool, table, lens, W ** -0.5), W, weight_error(Hq), "bad pages")
        err.zero_()
        out, lse = K.kamera_mla_attend_paged(pool.kv, LORA, q[:2].contiguous(), 16, table[:2].contiguous(), i32([301, -1]),
                                             300, err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == LEN and not bool(out.any()) and bool((lse == -float("inf")).all())


def test_decode_given_buffers_streams_and_graphs():
    lens = [700, 0, 129, 40]
    pool = Pool(7, 80, 16)
    table = pool.table(lens)
    pool.poison()
    q = normal(pool.g, 4, 16, W)
    args = (pool.kv, LORA, q, 16, table, i32(lens), 700)
    out, lse = K.kamera_mla_attend_paged(*args)
    need = K.kamera_mla_attend_paged_workspace_bytes(pool.kv, LORA, q, 16, 700)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)       # whatever it holds
    mine = torch.empty_like(out), torch.empty_like(lse)
    got = K.kamera_mla_attend_paged(*args, out=mine[0], lse=mine[1], workspace=ws)
    none = K.kamera_mla_attend_paged(*args, lse=False)
    torch.cuda.synchronize()
    assert got[0] is mine[0] and got[1] is mine[1] and none[1] is None
    assert torch.equal(out, mine[0]) and torch.equal(lse, mine[1]) and torch.equal(out, none[0])
    with pytest.raises(K.KameraError):
        K.kamera_mla_attend_paged(*args, workspace=ws[:-256])
    side = torch.cuda.Stream()
    a, b = K.kamera_mla_attend_paged(*args, stream=side)
    side.synchronize()
    assert torch.equal(a, out) and torch.equal(b, lse)
    graphs = []
    for _ in range(2):                                                  # two graphs, each with its own workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, K.kamera_mla_attend_paged(*args)))
    for _ in range(3):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, out) and torch.equal(b, lse) for _, (a, b) in graphs)


def test_decode_wait_runs_out_then_recovers(monkeypatch):
    for Hq in (16, 128):
        lens = [300, 65, 700]
        pool = Pool(8, 80, 16)
        table = pool.table(lens)
        q = normal(pool.g, 3, Hq, W)
        args = (pool.kv, LORA, q, 16, table, i32(lens), 700)
        good, _ = K.kamera_mla_attend_paged(*args)
        err = i32([0])
        monkeypatch.setenv("KAMERA_WAIT_LIMIT_NS", "1000000")
        monkeypatch.setenv("KAMERA_TEST_WITHHOLD_LOADS", "1")
        K.kamera_mla_attend_paged(*args, err=err)
        torch.cuda.synchronize()
        assert int(err.item()) & TIMEOUT
        monkeypatch.delenv("KAMERA_WAIT_LIMIT_NS")
        monkeypatch.delenv("KAMERA_TEST_WITHHOLD_LOADS")
        err.zero_()
        again, _ = K.kamera_mla_attend_paged(*args, err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0 and torch.equal(again, good)


# ----------------------------------------------------------------- expansion --
def expand_near(kv, pool, weight, slots):
    rows = R.f64(pool)[slots][:, :LORA]
    w = R.f64(weight)
    for h in range(w.shape[0]):
        ref = rows @ w[h].T
        tol = R.ulp_half(ref) + (1 + 2.0 ** -8) * 514 * 2.0 ** -24 * (np.abs(rows) @ np.abs(w[h]).T)
        assert np.all(np.abs(R.f64(kv[:, h]) - ref) <= tol), h


@pytest.mark.parametrize("T,H,pad", [(1, 1, 0), (127, 3, 8), (128, 16, 0), (129, 2, 16), (500, 5, 0), (1300, 16, 0)])
def test_expand_matches_definition(T, H, pad):
    g = gen(T)
    pool = normal(g, T + 40, W + pad)[:, :W]
    weight = normal(g, H, 256, LORA, std=0.05)
    slots = torch.randperm(T + 40, generator=g, device=DEV)[:T]
    err = i32([0])
    kv, kr = K.kamera_mla_expand(pool, LORA, weight, slots, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(kr, pool[slots][:, LORA:])
    expand_near(kv, pool, weight, slots.cpu().numpy())


def test_expand_padding_bad_slots_and_given_buffers():
    g = gen(1)
    pool, weight = normal(g, 50, W), normal(g, 2, 256, LORA, std=0.05)
    slots = torch.tensor([3, -1, 49, 3, -1] * 30, device=DEV)
    base = torch.full((150 * 2 * 256 + 8,), 7.0, dtype=BF, device=DEV)
    out = base[8:].view(150, 2, 256)                                    # 16-byte aligned, not 32
    kr = torch.full((150, 64), 7.0, dtype=BF, device=DEV)
    err = i32([0])
    a, b = K.kamera_mla_expand(pool, LORA, weight, slots, kv=out, k_rope=kr, err=err)
    torch.cuda.synchronize()
    assert a is out and b is kr and int(err.item()) == 0
    there = (slots >= 0).cpu().numpy()
    assert not bool(out[~torch.from_numpy(there).to(DEV)].any()) and not bool(kr[slots < 0].any())
    assert torch.equal(kr[slots >= 0], pool[slots[slots >= 0]][:, LORA:])
    expand_near(out[slots >= 0], pool, weight, slots.cpu().numpy()[there])
    assert bool((base[:8] == 7).all())
    for bad in (50, -2, 2 ** 40):
        slots[7] = bad
        err.zero_()
        kv, kr = K.kamera_mla_expand(pool, LORA, weight, slots, err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == SLOT and not bool(kv[7].any()) and not bool(kr[7].any())
    kv, kr = K.kamera_mla_expand(pool, LORA, weight, slots[:0])
    assert kv.shape == (0, 2, 256) and kr.shape == (0, 64)


def test_expand_wait_runs_out_then_recovers(monkeypatch):
    g = gen(2)
    pool, weight, slots = normal(g, 300, W), normal(g, 3, 256, LORA), torch.arange(300, device=DEV)
    good, _ = K.kamera_mla_expand(pool, LORA, weight, slots)
    err = i32([0])
    monkeypatch.setenv("KAMERA_WAIT_LIMIT_NS", "1000000")
    monkeypatch.setenv("KAMERA_TEST_WITHHOLD_LOADS", "1")
    K.kamera_mla_expand(pool, LORA, weight, slots, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) & TIMEOUT
    monkeypatch.delenv("KAMERA_WAIT_LIMIT_NS")
    monkeypatch.delenv("KAMERA_TEST_WITHHOLD_LOADS")
    again, _ = K.kamera_mla_expand(pool, LORA, weight, slots)
    torch.cuda.synchronize()
    assert torch.equal(again, good)


# ------------------------------------------------------------------- prefill --
def prefill_refs(q, kv, kr, qs, ks, scale, causal):
    """refs by (token, head), and the rows that some sequence has."""
    T, H = q.shape[:2]
    qf, kf, rf = R.f64(q), R.f64(kv), R.f64(kr)
    refs, seen = {}, []
    for s in range(len(qs) - 1):
        a, b, c, d = qs[s], qs[s + 1], ks[s], ks[s + 1]
        for h in range(H):
            k = np.concatenate([kf[c:d, h, :128], rf[c:d]], axis=1)
            for i, r in enumerate(L.prefill_rows(qf[a:b, h], k, kf[c:d, h, 128:], scale, causal)):
                refs[a + i, h] = r
        seen += list(range(a, b))
    return [refs[t, h] for t in seen for h in range(H)], seen


def starts(lens, gap=0):
    out = [gap]
    for n in lens:
        out.append(out[-1] + n)
    return out


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,nq,nk", [
    (1, [1], [1]), (2, [1, 5, 128, 0], [130, 5, 128, 9]), (3, [129, 255, 256, 257], [129, 300, 256, 513]),
    (2, [300, 7], [100, 3]), (1, [600], [1000]), (16, [33, 20], [33, 147]), (2, [140, 10], [0, 128]),
])
def test_prefill_matches_definition(H, nq, nk, causal):
    g = gen(H + sum(nq))
    qs, ks = starts(nq), starts(nk)
    q, kv, kr = normal(g, qs[-1], H, 192), normal(g, ks[-1], H, 256), normal(g, ks[-1], 64)
    err = i32([0])
    out, lse = K.kamera_mla_prefill_attend(q, kv, kr, i32(qs), i32(ks), max(nq), causal=causal, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    refs, _ = prefill_refs(q, kv, kr, qs, ks, 192 ** -0.5, causal)
    L.near(out, lse, refs, 192, 2.0 ** -8, (H, nq, nk, causal))


@pytest.mark.parametrize("causal", [True, False])
def test_prefill_of_many_blocks_matches_definition(causal):
    """More blocks of queries than two an SM: two blocks share the rows that a CTA reads."""
    g = gen(77)
    H, nq, nk = 18, [300, 1, 0, 257, 40, 3], [300, 131, 7, 400, 40, 260]
    qs, ks = starts(nq), starts(nk)
    q, kv, kr = normal(g, qs[-1], H, 192), normal(g, ks[-1], H, 256), normal(g, ks[-1], 64)
    out, lse = K.kamera_mla_prefill_attend(q, kv, kr, i32(qs), i32(ks), max(nq), causal=causal)
    torch.cuda.synchronize()
    refs, _ = prefill_refs(q, kv, kr, qs, ks, 192 ** -0.5, causal)
    L.near(out, lse, refs, 192, 2.0 ** -8, causal)


@pytest.mark.parametrize("scale", [-0.07, 0.0, 2.0])
def test_prefill_of_views_gaps_and_scales(scale):
    """Queries inside a wider projection, heads apart, rows with gaps of NaN between the
    sequences and behind them, keys that grow, outputs of rows that no sequence has."""
    g = gen(9)
    H, nq, nk = 3, [70, 200], [200, 131]
    wide = normal(g, 300, 5, 200)
    q = wide[:, 1:4, 8:]
    kvw, krw = normal(g, 420, H * 256 + 24), normal(g, 420, 80)
    kv, kr = kvw[:, :H * 256].unflatten(1, (H, 256)), krw[:, 16:]
    kv[:, :, :128] = (kv[:, :, :128].float() * torch.linspace(0.2, 3, 420, device=DEV)[:, None, None]).to(BF)
    qs, ks = starts(nq, 4), [11, 211, 342]
    kv[:11], kv[342:], kr[:11], kr[342:] = [float("nan")] * 4
    wide[:4], wide[4 + 270:] = float("nan"), float("nan")
    out = torch.full((300, H, 128), 5.0, dtype=BF, device=DEV)
    lse = torch.full((300, H), 5.0, device=DEV)
    a, b = K.kamera_mla_prefill_attend(q, kv, kr, i32(qs), i32(ks), 200, scale=scale, out=out, lse=lse)
    torch.cuda.synchronize()
    assert a is out and b is lse
    refs, seen = prefill_refs(q, kv, kr, qs, ks, float(np.float32(scale)), True)
    L.near(out[seen], lse[seen], refs, 192, 2.0 ** -8, scale)
    rest = [t for t in range(300) if t not in seen]
    assert bool((out[rest] == 5).all()) and bool((lse[rest] == 5).all())


def test_prefill_neighbours_of_nan_are_untouched():
    """A sequence whose rows are NaN leaves the others as they are."""
    g = gen(10)
    nq, nk = [100, 100, 50], [100, 150, 77]
    qs, ks = starts(nq), starts(nk)
    q, kv, kr = normal(g, 250, 2, 192), normal(g, 327, 2, 256), normal(g, 327, 64)
    ref, rl = K.kamera_mla_prefill_attend(q, kv, kr, i32(qs), i32(ks), 100)
    kv[100:250] = float("nan")
    out, lse = K.kamera_mla_prefill_attend(q, kv, kr, i32(qs), i32(ks), 100)
    torch.cuda.synchronize()
    for a, b in ((0, 100), (200, 250)):
        assert torch.equal(out[a:b], ref[a:b]) and torch.equal(lse[a:b], rl[a:b])
    assert bool(torch.isnan(out[100:200]).all())


@pytest.mark.parametrize("seqs,H", [(1, 2), (4, 40)])
def test_prefill_masked_values_that_are_not_finite(seqs, H):
    """A value that is not finite reaches the queries that see its row, in its column, and
    no other; so does a key (every column)."""
    g = gen(31)
    nq, nk = 270, 500                                          # query i sees rows up to i + 230
    qs, ks = starts([nq] * seqs), starts([nk] * seqs)
    q, kv, kr = normal(g, qs[-1], H, 192), normal(g, ks[-1], H, 256), normal(g, ks[-1], 64)
    args = (i32(qs), i32(ks), nq)
    ref, rl = K.kamera_mla_prefill_attend(q, kv, kr, *args)
    first = {}                                                 # (head, column) -> first row with one
    bad = kv.clone()
    for row, h, c, x in [(499, 0, 3, "nan"), (300, 0, 77, "inf"), (384, 0, 77, "inf"), (231, 1, 127, "-inf"),
                         (250, 1, 127, "inf"), (260, 1, 64, "nan"), (400, 0, 0, "-inf")]:
        bad[row, h, 128 + c] = float(x)
        first.setdefault((h, c), []).append((row, float(x)))
    out, lse = K.kamera_mla_prefill_attend(q, bad, kr, *args)
    torch.cuda.synchronize()
    assert torch.equal(lse, rl)
    want = ref.clone()
    for (h, c), rows in first.items():
        for row, x in rows:
            want[max(row - 230, 0):nq, h, c] += x              # (inf - inf: NaN)
    same = (out == want) | (out.isnan() & want.isnan())
    assert bool(same.all()), same.logical_not().nonzero()[:5]
    bad = kv.clone()
    bad[350, 1, 5] = float("nan")
    out, lse = K.kamera_mla_prefill_attend(q, bad, kr, *args)
    torch.cuda.synchronize()
    assert bool(out[120:nq, 1].isnan().all()) and bool(lse[120:nq, 1].isnan().all())
    out[120:nq, 1], lse[120:nq, 1] = ref[120:nq, 1], rl[120:nq, 1]
    assert torch.equal(out, ref) and torch.equal(lse, rl)


def test_prefill_reports_malformed_sequences():
    g = gen(11)
    q, kv, kr = normal(g, 60, 2, 192), normal(g, 80, 2, 256), normal(g, 80, 64)
    for qs, ks, mq, bit, good in (([0, 20, 60], [0, 81, 80], 40, DESCRIPTOR, []), ([0, 20, 61], [0, 30, 80], 60, DESCRIPTOR, [0]),
                                  ([-1, 20, 60], [0, 30, 80], 60, DESCRIPTOR, [1]), ([0, 20, 60], [0, 30, 80], 39, LEN, [0]),
                                  ([0, 20, 10], [0, 30, 80], 60, DESCRIPTOR, [0]), ([0, 20, 60], [40, 30, 80], 60, DESCRIPTOR, [1])):
        out, lse, err = torch.full((60, 2, 128), 5.0, dtype=BF, device=DEV), torch.full((60, 2), 5.0, device=DEV), i32([0])
        K.kamera_mla_prefill_attend(q, kv, kr, i32(qs), i32(ks), mq, out=out, lse=lse, err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == bit, (qs, ks)
        done = set()
        for s in good:
            a, b = qs[s], qs[s + 1]
            refs, _ = prefill_refs(q[a:b], kv, kr, [0, b - a], ks[s:s + 2], 192 ** -0.5, True)
            L.near(out[a:b], lse[a:b], refs, 192, 2.0 ** -8, (qs, ks))
            done |= set(range(a, b))
        rest = [t for t in range(60) if t not in done]
        assert bool((out[rest] == 5).all()) and bool((lse[rest] == 5).all()), (qs, ks)
    none = torch.zeros(0, 2, 192, dtype=BF, device=DEV)
    out, lse = K.kamera_mla_prefill_attend(none, kv, kr, i32([0]), i32([0]), 0)
    assert out.shape == (0, 2, 128)
    out, lse = K.kamera_mla_prefill_attend(q, kv[:0], kr[:0], i32([0, 60]), i32([0, 0]), 60)
    torch.cuda.synchronize()
    assert not bool(out.any()) and bool((lse == -float("inf")).all())


def test_prefill_wait_runs_out_then_recovers(monkeypatch):
    g = gen(12)
    q, kv, kr = normal(g, 400, 2, 192), normal(g, 500, 2, 256), normal(g, 500, 64)
    args = (q, kv, kr, i32([0, 10, 400]), i32([0, 70, 500]), 390)
    good, _ = K.kamera_mla_prefill_attend(*args)
    err = i32([0])
    monkeypatch.setenv("KAMERA_WAIT_LIMIT_NS", "1000000")
    monkeypatch.setenv("KAMERA_TEST_WITHHOLD_LOADS", "1")
    K.kamera_mla_prefill_attend(*args, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) & TIMEOUT
    monkeypatch.delenv("KAMERA_WAIT_LIMIT_NS")
    monkeypatch.delenv("KAMERA_TEST_WITHHOLD_LOADS")
    again, _ = K.kamera_mla_prefill_attend(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other, _ = K.kamera_mla_prefill_attend(*args, stream=side)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        third, _ = K.kamera_mla_prefill_attend(*args)
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, good) and torch.equal(other, good) and torch.equal(third, good)


# ------------------------------------------------------------------ together --
def test_prompt_and_decode_steps_together():
    """A prompt whose latent rows are appended, expanded and attended over, then decode
    steps that append a token and attend over the pool in the absorbed form: each against
    64-bit arithmetic on the rows that the pool holds.  Calls run without a wait between
    them, and once more with one, bit for bit the same."""
    H, P, n, prompt, steps = 4, 16, 2, [150, 37], 3
    inv = 1e4 ** (-2.0 * np.arange(32) / 64)
    rope = K.Rope(1e4, 64, 0, K.INTERLEAVED)

    def go(wait):
        g = gen(21)
        pool = torch.full((1, 24 * P, W), float("nan"), dtype=BF, device=DEV)
        order = torch.randperm(24, generator=g, device=DEV).tolist()
        table = [[order.pop() for _ in range(11)] for _ in range(n)]
        slot_of = lambda s, t: table[s][t // P] * P + t % P
        weight = normal(g, H, 256, LORA, std=LORA ** -0.5)
        qs = starts(prompt)
        T = qs[-1]
        c, kr, q = normal(g, T, LORA), normal(g, T, 64), normal(g, T, H, 192)
        slots = torch.tensor([slot_of(s, t) for s in range(n) for t in range(prompt[s])], device=DEV)
        pos = torch.tensor([t for s in range(n) for t in range(prompt[s])], device=DEV)
        err = i32([0])
        K.kamera_mla_append_kv(pool, LORA, c, kr, rope, pos, slots, q=q[:, :, 128:], q_out=q[:, :, 128:], err=err)
        wait()
        kv, k_rope = K.kamera_mla_expand(pool[0], LORA, weight, slots, err=err)
        wait()
        out, lse = K.kamera_mla_prefill_attend(q, kv, k_rope, i32(qs), i32(qs), max(prompt), scale=192 ** -0.5, err=err)
        wait()
        got, checks = [out, lse, kv, k_rope], [(q, kv, k_rope, qs)]
        for step in range(steps):
            c1, kr1, qn = normal(g, n, LORA), normal(g, n, 64), normal(g, n, H, 192)
            lens = [x + step + 1 for x in prompt]
            absorbed = torch.empty(n, H, W, dtype=BF, device=DEV)
            absorbed[:, :, :LORA] = torch.einsum("nhi,hic->nhc", qn[:, :, :128].float(), weight[:, :128].float()).to(BF)
            where = torch.tensor([slot_of(s, lens[s] - 1) for s in range(n)], device=DEV)
            K.kamera_mla_append_kv(pool, LORA, c1, kr1, rope, torch.tensor([x - 1 for x in lens], device=DEV), where,
                                   q=qn[:, :, 128:], q_out=absorbed[:, :, LORA:], err=err)
            wait()
            o, l = K.kamera_mla_attend_paged(pool[0], LORA, absorbed, P, i32(table), i32(lens), max(lens),
                                             scale=192 ** -0.5, err=err)
            wait()
            got += [o, l]
            checks.append((absorbed, lens))
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        return got, checks, pool, table, weight, slots, pos, kr

    got, checks, pool, table, weight, slots, pos, kr = go(lambda: None)
    alone = go(torch.cuda.synchronize)[0]
    assert all(torch.equal(a, b) for a, b in zip(got, alone))
    out, lse, kv, k_rope = got[:4]
    x = R.f64(kr)[:, None]
    ref = R.turned(x, pos.cpu().numpy(), inv, 0, True)
    tol = R.ulp_half(ref) + 2.0 ** -20 * (1 + 2.0 ** -8) * R.turn_scale(x, 32, 0, True)
    assert np.all(np.abs(R.f64(k_rope)[:, None] - ref) <= tol)
    expand_near(kv, pool[0], weight, slots.cpu().numpy())
    q, _, _, qs = checks[0]
    refs, _ = prefill_refs(q, kv, k_rope, qs, qs, float(np.float32(192 ** -0.5)), True)
    L.near(out, lse, refs, 192, 2.0 ** -8, "prompt")
    rows = R.f64(pool[0])
    for step in range(steps):
        absorbed, lens = checks[1 + step]
        refs = []
        for s in range(n):
            refs += L.latent_rows(R.f64(absorbed[s]), rows[R.slots_of(table[s], P, lens[s], 24)], LORA,
                                  float(np.float32(192 ** -0.5)))
        L.near(got[4 + 2 * step], got[5 + 2 * step], refs, W, 2.0 ** -16, ("step", step))
