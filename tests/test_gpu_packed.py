"""Pages in 4 bits: packing, unpacking and the attention that reads them, against their
definitions in 64 bits.  What packing stores is exact.  Attention's tolerance:
latent_ref.near with weights rounded to fp16 (2^-11, and smaller ones than 2^-21 of a
row's largest by 2^-32 of it), which also covers the tail's bf16 pairs (2^-16)."""
import numpy as np
import pytest
import torch

import position_invariant_kv_chunk_gb300 as K
from tests import latent_ref as L
from tests import paged_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
SLOT, LEN, TIMEOUT, VALUE = 1, 8, 32, 64
BF = torch.bfloat16
HALF, LEAST = 2.0 ** -11, 2.0 ** -32


def normal(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * std).to(BF)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def whole(n, P):
    return i32(list(range(n))), i32([P] * n)


def packed_like(n, H, P, d, fill=0):
    return torch.full((n, H, P * (d + d // 8)), fill, dtype=torch.uint8, device=DEV)


def pack_ref(k, v, P, n, ku=1.0, vu=1.0):
    """Pages 0 .. n-1 of pools [S, H, d] -> packed values, same shape, 64 bits."""
    k, v = R.f64(k), R.f64(v)
    pk, pv = np.zeros_like(k), np.zeros_like(v)
    for g in range(n):
        r = slice(g * P, g * P + P)
        pk[r], pv[r] = L.packed_page(k[r], v[r], ku, vu)
    return pk, pv


# --------------------------------------------------------------------- pages --
@pytest.mark.parametrize("H,d,P,units", [(4, 128, 16, (1.0, 1.0)), (1, 64, 48, (1.0, 0.25)), (3, 128, 64, (8.0, 2.0 ** -7)),
                                         (2, 64, 128, (2.0 ** -64, 2.0 ** 64)), (32, 128, 32, (0.5, 4.0))])
def test_packing_is_exact(H, d, P, units):
    g = gen(H + P)
    n = 5
    wide_k, wide_v = normal(g, n * P + 3, H * d + 8), normal(g, n * P + 3, H * d + 8)
    k, v = wide_k[:, :H * d].unflatten(1, (H, d)), wide_v[:, :H * d].unflatten(1, (H, d))
    k *= units[0]
    v *= units[1]
    k[:P] *= torch.exp(3 * torch.randn(P, H, d, generator=g, device=DEV)).to(BF)      # wide groups
    v[P:2 * P] *= torch.exp(3 * torch.randn(P, H, d, generator=g, device=DEV)).to(BF)
    packed = packed_like(n + 2, H, P, d)
    dst = i32([6, 0, 3, 1, 5])
    err = i32([0])
    assert K.kamera_pack_pages(k, v, P, i32([4, 3, 2, 1, 0]), i32([P] * 5), packed, dst, *units, err=err) is packed
    back_k, back_v = torch.full_like(wide_k, 3.0), torch.full_like(wide_v, 3.0)
    bk, bv = back_k[:, :H * d].unflatten(1, (H, d)), back_v[:, :H * d].unflatten(1, (H, d))
    K.kamera_unpack_pages(packed, P, dst, i32([P] * 5), bk, bv, i32([4, 3, 2, 1, 0]), *units, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    pk, pv = pack_ref(k, v, P, n, *units)
    assert np.array_equal(R.f64(bk)[:n * P], pk[:n * P]) and np.array_equal(R.f64(bv)[:n * P], pv[:n * P])
    assert bool((back_k[:, H * d:] == 3).all()) and bool((back_k[n * P:] == 3).all()) and bool((back_v[n * P:] == 3).all())


def test_packing_borders():
    """Every bf16 magnitude of some octaves beside a group maximum that makes the scale
    each of its fractions: numbers on borders between codes, and maxima on borders
    between scales, go where the definition says."""
    P, H, d = 16, 1, 128
    bits = torch.arange(0x3C00, 0x4180, device=DEV, dtype=torch.int32)         # 2^-7 .. 16
    values = bits.to(torch.int16).view(BF).float()
    tops = torch.tensor([6 * (1 + i / 16) * 2.0 ** e for i in range(16) for e in (-1, 0, 2)], device=DEV).to(BF)
    groups = []
    for t in tops.tolist():
        x = values[values <= t]
        x = x[:len(x) // 15 * 15].view(-1, 15)
        groups.append(torch.cat([torch.full((len(x), 1), t, device=DEV), x * (1 - 2 * (torch.arange(15, device=DEV) % 2))], 1))
    x = torch.cat(groups).to(BF)
    n = -(-len(x) // (P * d // 16))
    x = torch.cat([x, torch.zeros(n * P * d // 16 - len(x), 16, dtype=BF, device=DEV)])
    k = x.view(n * P, H, d).contiguous()
    v = x.view(n, d, 16).transpose(1, 2).reshape(n * P, H, d).contiguous()     # a channel's 16 tokens are a group
    packed, bk, bv = packed_like(n, H, P, d), torch.empty_like(k), torch.empty_like(v)
    ids, full = whole(n, P)
    K.kamera_pack_pages(k, v, P, ids, full, packed, ids)
    K.kamera_unpack_pages(packed, P, ids, full, bk, bv, ids)
    pk, pv = pack_ref(k, v, P, n)
    assert np.array_equal(R.f64(bk), pk) and np.array_equal(R.f64(bv), pv)


def test_packing_scale_of_every_maximum():
    """Every finite bf16 magnitude as a group's largest number, half of it and less beside."""
    P, H, d = 16, 1, 128
    x = torch.zeros(0x8000, 16, device=DEV)
    x[:0x7F80, 0] = torch.arange(0x7F80, device=DEV, dtype=torch.int32).to(torch.int16).view(BF).float()
    x[:, 1:] = x[:, :1] * (1 - 2 * (torch.arange(15, device=DEV) % 2)) * torch.linspace(0.01, 0.5, 15, device=DEV)
    x = x.to(BF)
    n = len(x) * 16 // (P * d)
    k = x.view(n * P, H, d).contiguous()
    v = x.view(n, d, 16).transpose(1, 2).reshape(n * P, H, d).contiguous()
    packed, bk, bv = packed_like(n, H, P, d), torch.empty_like(k), torch.empty_like(v)
    ids, full = whole(n, P)
    for units in ((1.0, 1.0), (2.0 ** -40, 2.0 ** 30)):
        K.kamera_pack_pages(k, v, P, ids, full, packed, ids, *units)
        K.kamera_unpack_pages(packed, P, ids, full, bk, bv, ids, *units)
        pk, pv = pack_ref(k, v, P, n, *units)
        assert np.array_equal(R.f64(bk), pk) and np.array_equal(R.f64(bv), pv), units


def test_packing_extremes():
    """Zeros, numbers too small for a scale, saturation, infinities, NaN."""
    P, H, d = 16, 2, 64
    g = gen(4)
    k, v = normal(g, P, H, d), normal(g, P, H, d)
    k[0, 0, :16] = 0.0
    k[1, 0, :16] = 2.0 ** -20
    k[2, 0, :16] = 1e30
    k[3, 0, 3] = float("inf")
    k[4, 1, 20] = -float("inf")
    v[:, 0, 5] = 3e4
    v[7, 1, 9] = -float("inf")
    k[5, 0, 16] = 6 * 2.0 ** -10                                # scale on the border to the least one: 0
    packed, bk, bv = packed_like(1, H, P, d), torch.empty_like(k), torch.empty_like(v)
    err = i32([0])
    one, full = whole(1, P)
    K.kamera_pack_pages(k, v, P, one, full, packed, one, err=err)
    K.kamera_unpack_pages(packed, P, one, full, bk, bv, one, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    pk, pv = pack_ref(k, v, P, 1)
    assert np.array_equal(R.f64(bk), pk) and np.array_equal(R.f64(bv), pv)
    assert R.f64(bk)[3, 0, 3] == 2688 and R.f64(bv)[7, 1, 9] == -2688
    k[6, 1, 33] = v[2, 0, 1] = float("nan")
    K.kamera_pack_pages(k, v, P, one, full, packed, one, err=err)
    K.kamera_unpack_pages(packed, P, one, full, bk, bv, one, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == VALUE
    pk, pv = pack_ref(k, v, P, 1)
    assert np.array_equal(R.f64(bk), pk) and np.array_equal(R.f64(bv), pv) and bk[6, 1, 33] == 0


def test_part_pages_and_errors():
    P, H, d = 48, 2, 128
    g = gen(6)
    n = 6
    k, v = normal(g, n * P, H, d), normal(g, n * P, H, d)
    counts = [48, 1, 16, 17, 0, 47]
    packed = packed_like(n, H, P, d, fill=0x5A)
    before = packed.clone()
    ids = i32(list(range(n)))
    err = i32([0])
    K.kamera_pack_pages(k, v, P, ids, i32(counts), packed, ids, err=err)
    bk, bv = torch.full_like(k, 9.0), torch.full_like(v, 9.0)
    K.kamera_unpack_pages(packed, P, ids, i32(counts), bk, bv, ids, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    piece = 18 * d
    kk, vv = k.clone(), v.clone()
    for i, c in enumerate(counts):
        pieces = -(-c // 16)
        assert torch.equal(packed[i, :, pieces * piece:], before[i, :, pieces * piece:])     # later tokens as they were
        kk[i * P + c:i * P + P], vv[i * P + c:i * P + P] = 0, 0
    pk, pv = pack_ref(kk, vv, P, n)
    for i, c in enumerate(counts):
        r, rest = slice(i * P, i * P + c), slice(i * P + c, i * P + P)
        assert np.array_equal(R.f64(bk)[r], pk[r]) and np.array_equal(R.f64(bv)[r], pv[r])
        assert bool((bk[rest] == 9).all()) and bool((bv[rest] == 9).all())
    before = packed.clone()
    for src, dst, c, bit in ((n, 0, 5, SLOT), (-1, 0, 5, SLOT), (0, n, 5, SLOT), (0, -7, 5, SLOT), (0, 1, 49, LEN),
                             (0, 1, -1, LEN)):
        err.zero_()
        K.kamera_pack_pages(k, v, P, i32([src]), i32([c]), packed, i32([dst]), err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == bit and torch.equal(packed, before), (src, dst, c)
        err.zero_()
        K.kamera_unpack_pages(packed, P, i32([dst]), i32([c]), bk, bv, i32([src]), err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == bit, (src, dst, c)
    K.kamera_pack_pages(k, v, P, ids[:0], ids[:0], packed, ids[:0])


# ----------------------------------------------------------------- attention --
class Cache:
    """Sequences with a packed part and a bf16 tail.  Bytes that nothing wrote are 0xFF
    (scales that are NaN as fp16), rows that no table names NaN."""

    def __init__(self, seed, lens, tails, H, d, P, TP=None, units=(1.0, 1.0), grow=False):
        self.g, self.P, self.TP, self.H, self.d, self.units = gen(seed), P, TP or P, H, d, units
        self.lens, self.tails = lens, tails
        n = sum(-(-x // P) for x in lens)
        k, v = normal(self.g, max(n, 1) * P, H, d, std=units[0]), normal(self.g, max(n, 1) * P, H, d, std=units[1])
        if grow:
            k = (k.float() * torch.linspace(0.1, 4, len(k), device=DEV)[:, None, None]).to(BF)
        self.n = n + 3
        self.packed = packed_like(self.n, H, P, d, fill=0xFF)
        order = torch.randperm(self.n, generator=self.g, device=DEV).tolist()
        src, dst, count, self.rows = [], [], [], []
        for x in lens:
            first, mine = len(src), []
            for j in range(-(-x // P)):
                src.append(first + j)
                mine.append(order.pop())
                count.append(min(P, x - j * P))
            dst += mine
            self.rows.append((first, mine))
        if n:
            K.kamera_pack_pages(k, v, P, i32(src), i32(count), self.packed, i32(dst), *units)
        for i, c in enumerate(count):
            k[i * P + c:i * P + P], v[i * P + c:i * P + P] = 0, 0
        self.pk, self.pv = pack_ref(k, v, P, n, *units)
        width = max([len(m) for _, m in self.rows] + [1])
        self.table = i32([m + [2 ** 31 - 1] * (width - len(m)) for _, m in self.rows])
        tn = [-(-x // self.TP) for x in tails]
        self.tk, self.tv = normal(self.g, (sum(tn) + 2) * self.TP, H, d), normal(self.g, (sum(tn) + 2) * self.TP, H, d)
        order = torch.randperm(sum(tn) + 2, generator=self.g, device=DEV).tolist()
        tt = [[order.pop() for _ in range(c)] for c in tn]
        self.tail_table = i32([m + [-5] * (max(tn + [1]) - len(m)) for m in tt])
        self.tail_slots = [R.slots_of(m, self.TP, x, sum(tn) + 2) for m, x in zip(tt, tails)]
        used = torch.zeros(len(self.tk), dtype=torch.bool, device=DEV)
        for s in self.tail_slots:
            used[torch.from_numpy(s).to(DEV)] = True
        self.tk[~used] = float("nan")
        self.tv[~used] = float("nan")

    def args(self, q, tail=True):
        a = (self.packed, q, self.P, self.table, i32(self.lens), max(self.lens))
        return a + ((self.tk, self.tv, self.tail_table, i32(self.tails), max(self.tails), self.TP) if tail else ())

    def refs(self, q, scale, tail=True, left_out=()):
        """left_out: (sequence, place in its page table) of pages that do not count."""
        qf, out = R.f64(q), []
        G = q.shape[1] // self.H
        tk, tv = R.f64(self.tk), R.f64(self.tv)
        for s, n in enumerate(self.lens):
            first, _ = self.rows[s]
            t = np.arange(n)
            t = t[[(s, j) not in left_out for j in t // self.P]] if left_out else t
            at = first * self.P + t
            ts = self.tail_slots[s] if tail else np.zeros(0, dtype=int)
            for h in range(self.H):
                k = np.concatenate([self.pk[at, h], tk[ts, h]])
                v = np.concatenate([self.pv[at, h], tv[ts, h]])
                o, l, m, x = R.attention(qf[s, h * G:h * G + G], k, v, scale)
                out += [(o[g], l[g], m[g], x[g], len(k), np.abs(v).sum(0)) for g in range(G)]
        return out


@pytest.mark.parametrize("H,G,d,P,TP", [(4, 7, 128, 16, 16), (2, 8, 64, 48, 16), (1, 1, 128, 64, 32), (3, 16, 128, 32, 64),
                                        (2, 9, 64, 16, 16), (8, 4, 64, 128, 16), (32, 1, 128, 16, 16)])
def test_attention_matches_definition(H, G, d, P, TP):
    lens = [0, 1, 15, 127, 128, 129, 500, 0]
    tails = [5, 0, 17, 1, 16, 70, 3, 0]
    c = Cache(H + G, lens, tails, H, d, P, TP)
    q = normal(c.g, len(lens), H * G, d)
    err = i32([0])
    out, lse = K.kamera_attend_packed(*c.args(q), err=err)
    alone = K.kamera_attend_packed(*c.args(q, tail=False), err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    L.near(out, lse, c.refs(q, d ** -0.5), d, HALF, "with tails", LEAST)
    L.near(*alone, c.refs(q, d ** -0.5, tail=False), d, HALF, "packed alone", LEAST)


@pytest.mark.parametrize("lens", [[20000], [int(x) for x in np.random.default_rng(3).integers(0, 60, 300)], [0] * 4, [3000] * 9])
def test_attention_of_one_long_and_many_short(lens):
    tails = [(7 * i) % 40 for i in range(len(lens))]
    c = Cache(len(lens), lens, tails, 2, 128, 16)
    q = normal(c.g, len(lens), 8, 128)
    out, lse = K.kamera_attend_packed(*c.args(q))
    L.near(out, lse, c.refs(q, 128 ** -0.5), 128, HALF, len(lens), LEAST)


@pytest.mark.parametrize("scale,units,qs", [(0.3, (1.0, 1.0), 1.0), (-0.1, (1.0, 1.0), 1.0), (0.0, (1.0, 1.0), 1.0),
                                            (0.05, (16.0, 2.0 ** -9), 1.0), (2.0 ** 20, (1.0, 1.0), 2.0 ** -22),
                                            (2.0 ** -40, (1.0, 1.0), 2.0 ** 38)])
@pytest.mark.parametrize("G", [5, 12])
def test_attention_of_growing_scores_scales_and_units(scale, units, qs, G):
    """Keys that grow along the sequence move the running maximum; negative and zero
    scales, units, and queries of extreme size (their power of two is taken out)."""
    d = 64
    c = Cache(17, [700, 300], [20, 0], 2, d, 16, units=units, grow=True)
    q = normal(c.g, 2, 2 * G, d, std=qs)
    q[0, 1] = 0.0
    out, lse = K.kamera_attend_packed(*c.args(q), scale=scale, k_unit=units[0], v_unit=units[1])
    L.near(out, lse, c.refs(q, float(np.float32(scale))), d, HALF, (scale, units, qs), LEAST)


def test_attention_reports_bad_pages_and_lengths():
    c = Cache(23, [600, 100, 128, 16], [10, 0, 4, 0], 2, 128, 16)
    q = normal(c.g, 4, 8, 128)
    c.table[0, 2], c.table[0, 8:20], c.table[1, 6], c.table[3, 0] = -1, c.n, 2 ** 31 - 1, -9
    out_of = {(0, 2), (1, 6), (3, 0)} | {(0, j) for j in range(8, 20)}
    err = i32([0])
    out, lse = K.kamera_attend_packed(*c.args(q), err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == SLOT
    L.near(out, lse, c.refs(q, 128 ** -0.5, left_out=out_of), 128, HALF, "bad pages", LEAST)
    err.zero_()
    c = Cache(24, [64, 30], [0, 0], 2, 128, 16)
    q = normal(c.g, 2, 8, 128)
    out, lse = K.kamera_attend_packed(c.packed, q, 16, c.table, i32([65, -3]), 64, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == LEN and not bool(out.any()) and bool((lse == -float("inf")).all())


def test_attention_given_buffers_streams_and_graphs():
    c = Cache(25, [900, 0, 130], [20, 3, 0], 4, 128, 16)
    q = normal(c.g, 3, 28, 128)
    out, lse = K.kamera_attend_packed(*c.args(q))
    need = K.kamera_attend_packed_workspace_bytes(c.packed, q, 16, 900, 20)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    mine = torch.empty_like(out), torch.empty_like(lse)
    got = K.kamera_attend_packed(*c.args(q), out=mine[0], lse=mine[1], workspace=ws)
    none = K.kamera_attend_packed(*c.args(q), lse=False)
    torch.cuda.synchronize()
    assert got[0] is mine[0] and got[1] is mine[1] and none[1] is None
    assert torch.equal(out, mine[0]) and torch.equal(lse, mine[1]) and torch.equal(out, none[0])
    with pytest.raises(K.KameraError):
        K.kamera_attend_packed(*c.args(q), workspace=ws[:-256])
    side = torch.cuda.Stream()
    a, b = K.kamera_attend_packed(*c.args(q), stream=side)
    side.synchronize()
    assert torch.equal(a, out) and torch.equal(b, lse)
    args, graphs = c.args(q), []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, K.kamera_attend_packed(*args)))
    for _ in range(3):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, out) and torch.equal(b, lse) for _, (a, b) in graphs)


def test_attention_wait_runs_out_then_recovers(monkeypatch):
    c = Cache(26, [900, 400], [20, 30], 2, 128, 16)
    q = normal(c.g, 2, 14, 128)
    good, _ = K.kamera_attend_packed(*c.args(q))
    err = i32([0])
    monkeypatch.setenv("KAMERA_WAIT_LIMIT_NS", "1000000")
    monkeypatch.setenv("KAMERA_TEST_WITHHOLD_LOADS", "1")
    K.kamera_attend_packed(*c.args(q, tail=False), err=err)
    torch.cuda.synchronize()
    assert int(err.item()) & TIMEOUT
    monkeypatch.delenv("KAMERA_WAIT_LIMIT_NS")
    monkeypatch.delenv("KAMERA_TEST_WITHHOLD_LOADS")
    err.zero_()
    again, _ = K.kamera_attend_packed(*c.args(q), err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(again, good)


# ------------------------------------------------------------------ together --
def test_decode_steps_that_pack_full_pages():
    """Decode steps that append a token, pack the page that has filled and attend over
    packed pages and tail, without a wait between the calls: each step against 64-bit
    arithmetic on what both pools hold, and once more with waits, bit for bit the same;
    unpacked pages read by attention over the bf16 pool give the same rows."""
    H, G, d, P, n, steps = 2, 7, 128, 16, 3, 2 * 16 + 5
    rope = K.Rope(1e4, d)

    def go(wait):
        g = gen(31)
        pool = [normal(g, 1, 8 * P, H, d), normal(g, 1, 8 * P, H, d)]
        packed = packed_like(n * 4, H, P, d, fill=0xFF)
        start = [5, 0, 11]                                        # tokens already in the page being filled
        length, done = list(start), [0] * n
        got, states, err = [], [], i32([0])
        for _ in range(steps):
            k, v, q = normal(g, n, H, d), normal(g, n, H, d), normal(g, n, H * G, d)
            slots = torch.tensor([s * P + length[s] % P for s in range(n)], device=DEV)   # a sequence's page: s
            pos = torch.tensor(length, device=DEV)
            turned = K.kamera_append_kv(*pool, k, v, rope, pos, slots, q=q, err=err)
            wait()
            length = [x + 1 for x in length]
            full = [s for s in range(n) if length[s] % P == 0]
            if full:
                K.kamera_pack_pages(pool[0][0], pool[1][0], P, i32(full), i32([P] * len(full)), packed,
                                    i32([4 * s + done[s] for s in full]), err=err)
                wait()
                for s in full:
                    done[s] += 1
            lens, tails = [P * x for x in done], [x - P * y for x, y in zip(length, done)]
            table = i32([[4 * s + j for j in range(4)] for s in range(n)])
            out, lse = K.kamera_attend_packed(packed, turned, P, table, i32(lens), max(lens), pool[0][0], pool[1][0],
                                              i32([[s] for s in range(n)]), i32(tails), max(tails), err=err)
            wait()
            got += [out, lse]
            states.append((turned, lens, tails, pool[0][0, :n * P].clone(), pool[1][0, :n * P].clone(), list(done)))
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        return got, states, packed

    got, states, packed = go(lambda: None)
    alone = go(torch.cuda.synchronize)[0]
    assert all(torch.equal(a, b) for a, b in zip(got, alone))
    pages = 4 * n
    bk, bv = torch.zeros(pages * P, H, d, dtype=BF, device=DEV), torch.zeros(pages * P, H, d, dtype=BF, device=DEV)
    done = states[-1][-1]
    filled = [4 * s + j for s in range(n) for j in range(done[s])]
    K.kamera_unpack_pages(packed, P, i32(filled), i32([P] * len(filled)), bk, bv, i32(filled))
    torch.cuda.synchronize()
    pk, pv = R.f64(bk), R.f64(bv)
    for i in list(range(0, steps, 6)) + [steps - 1]:
        turned, lens, tails, tk, tv, _ = states[i]
        qf, tk, tv, refs = R.f64(turned), R.f64(tk), R.f64(tv), []
        for s in range(n):
            a, b = slice(4 * s * P, 4 * s * P + lens[s]), slice(s * P, s * P + tails[s])
            for h in range(H):
                o, l, m, x = R.attention(qf[s, h * G:h * G + G], np.concatenate([pk[a, h], tk[b, h]]),
                                         np.concatenate([pv[a, h], tv[b, h]]), d ** -0.5)
                refs += [(o[j], l[j], m[j], x[j], lens[s] + tails[s],
                          np.abs(pv[a, h]).sum(0) + np.abs(tv[b, h]).sum(0)) for j in range(G)]
        L.near(got[2 * i], got[2 * i + 1], refs, d, HALF, ("step", i), LEAST)
    turned, lens = states[-1][:2]
    table = i32([[4 * s + j for j in range(4)] for s in range(n)])
    a, al = K.kamera_attend_shared(bk, bv, turned, P, None, None, None, table, i32(lens), 0, 0, max(lens))
    qf, refs = R.f64(turned), []
    for s in range(n):
        r = slice(4 * s * P, 4 * s * P + lens[s])
        for h in range(H):
            o, l, m, x = R.attention(qf[s, h * G:h * G + G], pk[r, h], pv[r, h], d ** -0.5)
            refs += [(o[j], l[j], m[j], x[j], lens[s], np.abs(pv[r, h]).sum(0)) for j in range(G)]
    b, bl = K.kamera_attend_packed(packed, turned, P, table, i32(lens), max(lens))
    L.near(a, al, refs, d, 2.0 ** -16, "unpacked")
    L.near(b, bl, refs, d, HALF, "packed", LEAST)
