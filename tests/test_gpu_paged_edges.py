"""Decode steps over the paged pool at their edges.  Tolerances are those of
test_gpu_append and test_gpu_paged.  (There a weight's split counts 2^-17 in numerator and
denominator; hi rounded towards zero and lo to nearest are off by 2^-16, in the
numerator alone: the same sum.)"""
import numpy as np
import pytest
import torch

import position_invariant_kv_chunk_gb300 as K
from tests import paged_ref as R
from tests.test_gpu_paged import DEV, Pool, boxes, i32, near, normal, rows_ref, select_ref

pytestmark = pytest.mark.gpu
SLOT, DESCRIPTOR, TIMEOUT = 1, 4, 32


# ------------------------------------------------------------------- append --
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_of_negative_frequencies_is_the_mirror_image(interleaved):
    """R(p) at -theta is R(-p) at theta, bit for bit, out to the ends of the position
    range: phases are whole numbers, and both forms make the same ones."""
    T, H, d = 1500, 2, 128
    g = torch.Generator(device=DEV).manual_seed(61)
    k, v = normal(g, T, H, d), normal(g, T, H, d)
    pos = torch.randint(2 ** 30, 2 ** 31 - 1, (T,), generator=g, device=DEV)
    pos[::2] *= -1
    pos[0], pos[1] = 2 ** 31 - 1, -(2 ** 31 - 1)
    inv = 1e6 ** (-2.0 * np.arange(d // 2) / d)
    got = []
    for sign in (1, -1):
        pk, pv = torch.zeros(1, T, H, d, dtype=torch.bfloat16, device=DEV), torch.zeros(1, T, H, d, dtype=torch.bfloat16,
                                                                                         device=DEV)
        rope = K.Rope(1e6, d, 0, K.INTERLEAVED if interleaved else K.ROTATE_HALF, inv_freq=sign * inv)
        K.kamera_append_kv(pk, pv, k, v, rope, sign * pos, torch.arange(T, device=DEV))
        got.append(pk)
    torch.cuda.synchronize()
    assert torch.equal(got[0], got[1])


# ---------------------------------------------------------------- selection --
def cancelling_boxes(gen, n, d):
    """Boxes of one point whose large even channels cancel in pairs against a query of
    ones: what is left of a score is its channel 7, a whole number below 256 times 2^-12,
    which fp32 sums lose beside terms of up to 2^20."""
    x = torch.zeros(n, d, dtype=torch.bfloat16, device=DEV)
    big = normal(gen, n, d // 4).float() * 2.0 ** torch.randint(0, 20, (n, d // 4), generator=gen, device=DEV)
    x[:, 0::4], x[:, 2::4] = big.to(torch.bfloat16), -big.to(torch.bfloat16)
    x[:, 7] = ((torch.randperm(n, generator=gen, device=DEV) % 251).float() * 2.0 ** -12).to(torch.bfloat16)
    return torch.stack([x, x], dim=1)[:, None].contiguous()


@pytest.mark.parametrize("d,width", [(128, 400), (64, 400), (128, 2600)])
def test_selection_beside_a_nan_box(d, width):
    """A box with a NaN in one even channel, in every sixteen pages: it comes first, and
    the order of the pages beside it, whose scores fp32 cannot tell apart, stays exact."""
    P, k = 16, 30 + width // 16
    g = torch.Generator(device=DEV).manual_seed(71)
    summary = cancelling_boxes(g, width, d)
    summary[6::16, 0, :, 4] = float("nan")
    q = torch.ones(1, 1, d, dtype=torch.bfloat16, device=DEV)
    pages = torch.arange(width, device=DEV, dtype=torch.int32)[None]
    got = K.kamera_select_pages(q, summary, P, pages, i32([width * P]), width * P, k)
    torch.cuda.synchronize()
    assert np.array_equal(got.cpu().numpy(), select_ref(q, summary, pages, [width * P], P, k, 1, 1))


@pytest.mark.parametrize("d,width", [(128, 400), (64, 400), (128, 2600), (64, 2600)])
def test_selection_with_infinite_bounds_that_no_query_asks_for(d, width):
    """A minimum of -infinity where every query is positive, a maximum of infinity where
    every query is negative: the score is finite, and the page takes its place by it.
    Infinities on the side that counts still come first."""
    H, G, P, n = 2, 3, 16, 2
    g = torch.Generator(device=DEV).manual_seed(72)
    summary = boxes(g, width, H, d)
    sign = torch.where(torch.arange(d, device=DEV) % 3 == 0, -1.0, 1.0)
    q = ((normal(g, n, H * G, d).abs() + 0.25) * sign).to(torch.bfloat16)
    summary[2::5, :, 0, 10] = -float("inf")
    summary[3::7, 1, 1, 9] = float("inf")
    summary[4::11, 0, 0, 1] = -float("inf")
    summary[101, 0, 1, 10] = float("inf")
    lens = [width * P, (width - 70) * P]
    pages = torch.stack([torch.randperm(width, generator=g, device=DEV) for _ in lens]).to(torch.int32)
    for k in (5, width // 3):
        got = K.kamera_select_pages(q, summary, P, pages, i32(lens), max(lens), k)
        torch.cuda.synchronize()
        ref = select_ref(q, summary, pages, lens, P, k, 1, 1)
        assert np.array_equal(got.cpu().numpy(), ref), k


@pytest.mark.parametrize("d,width", [(128, 400), (64, 400), (128, 2600)])
def test_selection_beside_infinite_bounds(d, width):
    """Pages that fp32 cannot tell apart, with a bound of -infinity that counts for
    nothing among every sixteen of them."""
    P, k = 16, 30 + width // 16
    g = torch.Generator(device=DEV).manual_seed(73)
    summary = cancelling_boxes(g, width, d)
    summary[9::16, 0, 0, 4] = -float("inf")
    q = torch.ones(1, 1, d, dtype=torch.bfloat16, device=DEV)
    pages = torch.randperm(width, generator=g, device=DEV)[None].to(torch.int32)
    got = K.kamera_select_pages(q, summary, P, pages, i32([width * P]), width * P, k)
    torch.cuda.synchronize()
    assert np.array_equal(got.cpu().numpy(), select_ref(q, summary, pages, [width * P], P, k, 1, 1))


# ---------------------------------------------------------------- attention --
@pytest.mark.parametrize("P,cut", [(1024, 0), (1024, 1000), (16, 5)])
def test_selected_attention_of_lengths_near_2_31(P, cut):
    """A sequence of nearly 2^31 tokens over a few pages: its last pages are inside it."""
    H, G, d, n = 1, 4, 64, 0x7FFFFF00 - cut
    if P == 16:
        n = 1 << 27                                   # (the table of shorter pages)
    pool = Pool(81, 6, P, H, d)
    width = -(-n // P)
    table = (torch.arange(width, device=DEV) % 6).to(torch.int32)[None]
    q = normal(pool.g, 1, H * G, d)
    chosen = [0, 7, width - 2, width - 1]
    sel = i32([[chosen]])
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = K.kamera_attend_selected(pool.k, pool.v, q, P, table, i32([n]), sel, n, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    slots = np.concatenate([np.arange(j % 6 * P, j % 6 * P + min(P, n - j * P)) for j in chosen])
    idx = torch.from_numpy(slots).to(DEV)
    o, l, m, x = R.attention(R.f64(q)[0], R.f64(pool.k[idx])[:, 0], R.f64(pool.v[idx])[:, 0], d ** -0.5)
    near(out, lse, [(o[g], l[g], m[g], x[g], len(slots)) for g in range(G)], "long")
    K.kamera_attend_selected(pool.k, pool.v, q, P, table, i32([n - P]), sel, n, err=err)   # the last page is past it
    torch.cuda.synchronize()
    assert int(err.item()) == 1


def special(pool, rows, values):
    """Sets pool.v[row, head, channel] to the values; rows, values: ((row, head, channel), value) pairs."""
    for (r, h, c), x in zip(rows, values):
        pool.v[r, h, c] = x


def near_with_infinities(out, lse, q, pool, slot_lists, scale, what):
    """Each channel with an infinite value of one sign is that infinity, with both signs
    or a NaN it is NaN, and every other one is within the tolerance; an infinite value
    whose weight fp32 rounds to nothing (zero times infinity) may leave NaN.  slot_lists[s][h]."""
    n, hq, d = q.shape
    G = hq // pool.H
    got, qh, refs = out.clone().view(n, pool.H, G, d), R.f64(q), []
    for s in range(n):
        for h in range(pool.H):
            idx = torch.from_numpy(slot_lists[s][h]).to(DEV)
            kk, vv = R.f64(pool.k[idx])[:, h], R.f64(pool.v[idx])[:, h]
            up, down, nan = np.isposinf(vv).any(0), np.isneginf(vv).any(0), np.isnan(vv).any(0)
            nan |= up & down
            mine = R.f64(got[s, h])
            assert np.isnan(mine[:, nan]).all(), what
            if len(idx):                            # weights relative to each row's largest, in powers of two
                z = scale * 1.4426950408889634 * (qh[s, h * G:h * G + G] @ kk.T)
                some = (z - z.max(1, keepdims=True) > -100)[:, :, None] | ~np.isinf(vv)
                full = some.all(1)                  # [G, d]: every infinite value has weight
                assert not np.isfinite(mine[:, up | down]).any(), what
                assert np.isposinf(mine[full & (up & ~nan)]).all(), what
                assert np.isneginf(mine[full & (down & ~nan)]).all(), what
            off = torch.from_numpy(up | down | nan).to(DEV)
            got[s, h, :, off] = 0
            vv[:, up | down | nan] = 0
            o, l, m, x = R.attention(qh[s, h * G:h * G + G], kk, vv, scale)
            refs += [(o[g], l[g], m[g], x[g], len(idx)) for g in range(G)]
    near(got.view(n, hq, d), lse, refs, what)


INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("H,G,d,P,prefix,lens", [
    (2, 7, 128, 16, 700, [50, 333, 0]),        # prefix and own pages, one side of the prefix kernel
    (32, 2, 128, 16, 1300, [50, 33]),
    (3, 16, 64, 32, 2000, [5, 70, 1, 40] * 6),  # two tiles of rows
    (1, 3, 64, 16, 0, [700, 1, 33]),           # own pages, joined in a cluster
    (2, 9, 128, 16, 0, [20, 4000]),            # in a cluster of several CTAs
    (2, 4, 64, 16, 0, [30000, 17]),            # through the workspace
])
def test_shared_infinite_values(H, G, d, P, prefix, lens):
    n = len(lens)
    pool = Pool(91 + H + G, -(-prefix // P) + sum(-(-x // P) for x in lens) + 3, P, H, d)
    pre, own = pool.table([prefix]), pool.table(lens)
    pool.poison()
    q = normal(pool.g, n, H * G, d)
    q[:, :, 0] = 4.0
    a = R.slots_of(pre[0].tolist(), P, prefix, pool.n_pages)
    b = [R.slots_of(own[s].tolist(), P, x, pool.n_pages) for s, x in enumerate(lens)]
    long = int(np.argmax(lens))
    first = b[long]
    pool.k[int(first[1]), :, 0] = -60.0            # a weight that fp32 rounds to nothing
    special(pool, [(int(first[1]), 0, 2), (int(first[0]), H - 1, 3), (int(first[-1]), 0, 5), (int(first[2]), 0, 5),
                   (int(first[3]), 0, d - 1), (int(first[4]), H - 1, 9), (int(first[16]), 0, 40)],
            [INF, -INF, INF, -INF, -INF, NAN, INF])
    if prefix:
        pool.k[int(a[290]), :, 0] = -60.0
        special(pool, [(int(a[0]), 0, 17), (int(a[prefix - 1]), H - 1, 20), (int(a[290]), 0, d - 3),
                       (int(a[150]), 0, 33), (int(a[160]), 0, 33), (int(first[0]), 0, 17)],
                [INF, -INF, -INF, INF, -INF, -INF])
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    if prefix:
        out, lse = K.kamera_attend_shared(pool.k, pool.v, q, P, i32([0, n]), pre, i32([prefix]), own, i32(lens), n,
                                          prefix, max(lens), err=err)
    else:
        out, lse = K.kamera_attend_shared(pool.k, pool.v, q, P, None, None, None, own, i32(lens), 0, 0, max(lens),
                                          err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    near_with_infinities(out, lse, q, pool, [[np.concatenate([a, b[s]])] * H for s in range(n)], d ** -0.5, (H, G, d))


@pytest.mark.parametrize("k,G", [(6, 3), (300, 8)])
def test_selected_infinite_values(k, G):
    """Infinite values in selected pages count, those in other pages do not."""
    H, d, P, lens = 2, 128, 16, [9000, 100]
    pool = Pool(95, sum(-(-x // P) for x in lens) + 2, P, H, d)
    pages = pool.table(lens)
    pool.poison()
    q = normal(pool.g, 2, H * G, d)
    rng = np.random.default_rng(7)
    sel = torch.full((2, H, k), -1, dtype=torch.int32, device=DEV)
    for s in range(2):
        count = -(-lens[s] // P)
        for h in range(H):
            take = np.sort(rng.permutation(count)[:k])
            sel[s, h, :len(take)] = torch.from_numpy(take).to(DEV)
    slots = [R.slots_of(pages[s].tolist(), P, x, pool.n_pages) for s, x in enumerate(lens)]
    for s in range(2):
        for j in range(0, lens[s], 37):
            pool.v[int(slots[s][j]), j % H, j % d] = INF if j % 2 else -INF
    out, lse = K.kamera_attend_selected(pool.k, pool.v, q, P, pages, i32(lens), sel, max(lens))
    torch.cuda.synchronize()
    lists = [[np.concatenate([slots[s][j * P:j * P + P] for j in sel[s, h].tolist() if j >= 0]) for h in range(H)]
             for s in range(2)]
    near_with_infinities(out, lse, q, pool, lists, d ** -0.5, k)


def test_one_head_of_any_head_stride():
    """A pool of one KV head whose head stride is no row's: appended to and attended over."""
    S, d, P, T, Hq = 64, 64, 16, 20, 3
    g = torch.Generator(device=DEV).manual_seed(97)
    view = lambda x: x.as_strided((1, S, 1, d), (5, d, 40, 1))
    pk, pv = view(normal(g, S * d)), view(normal(g, S * d))
    k, v, q = normal(g, T, 1, d), normal(g, T, 1, d), normal(g, 1, Hq, d)
    slots = torch.randperm(S, generator=g, device=DEV)[:T].contiguous()
    pk2, pv2 = pk.clone(memory_format=torch.contiguous_format), pv.clone(memory_format=torch.contiguous_format)
    table, lens = i32([[2, 0, 3]]), i32([41])
    got = []
    for a, b in ((pk, pv), (pk2, pv2)):
        K.kamera_append_kv(a, b, k, v, K.Rope(1e4, d), torch.arange(T, device=DEV), slots)
        got.append(K.kamera_attend_shared(a[0], b[0], q, P, None, None, None, table, lens, 0, 0, 41))
    torch.cuda.synchronize()
    assert torch.equal(pk, pk2) and torch.equal(pv, pv2)
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_workspaces_of_the_size_that_is_given():
    """A workspace of exactly the bytes that Python names is enough, one less is refused."""
    H, G, d, P, lens = 2, 7, 128, 16, [700, 33]
    pool = Pool(98, 120, P, H, d)
    pre, own = pool.table([600]), pool.table(lens)
    pool.poison()
    q = normal(pool.g, 2, H * G, d)
    summary, select = boxes(pool.g, 120, H, d), i32([[list(range(43))] * H] * 2)
    calls = [
        (K.kamera_attend_shared_workspace_bytes(pool.k, q, P, 1, 2, 600, 700),
         lambda **w: K.kamera_attend_shared(pool.k, pool.v, q, P, i32([0, 2]), pre, i32([600]), own, i32(lens), 2, 600, 700,
                                            **w)[0]),
        (K.kamera_select_pages_workspace_bytes(q, summary, P, 700, 9),
         lambda **w: K.kamera_select_pages(q, summary, P, own, i32(lens), 700, 9, **w)),
        (K.kamera_attend_selected_workspace_bytes(pool.k, q, P, 43, 700),
         lambda **w: K.kamera_attend_selected(pool.k, pool.v, q, P, own, i32(lens), select, 700, **w)[0]),
    ]
    assert [n > 0 for n, _ in calls] == [True, True, False]     # the last one's splits join in a cluster
    for n, call in calls:
        room = torch.empty(n, dtype=torch.uint8, device=DEV)
        assert torch.equal(call(), call(workspace=room))
        if n:
            with pytest.raises(K.KameraError):
                call(workspace=room[:n - 1])
    torch.cuda.synchronize()


# --------------------------------------- prefixes whose tiles go to the sides in turn
class InTurn:
    """Enough (group, KV head) pairs that every prefix stays in one piece, of 128 rows at
    most and eight tiles at least: the prefix kernel's two sides take its tiles in turn."""

    def __init__(self, seed, H, G, d, P, groups, prefix, lens, std=1.0):
        self.P, self.G, self.prefix, self.lens = P, G, prefix, lens
        n = sum(groups)
        need = sum(-(-x // P) for x in prefix + lens) + 3
        self.pool = Pool(seed, need, P, H, d, std=std)
        self.pre, self.own = self.pool.table(prefix), self.pool.table(lens)
        self.pool.poison()
        self.q = normal(self.pool.g, n, H * G, d)
        self.starts = np.concatenate([[0], np.cumsum(groups)])
        self.args = (i32(self.starts.tolist()), self.pre, i32(prefix), self.own, i32(lens), max(groups), max(prefix),
                     max(lens))
        rows = n * H * G
        align = lambda x: -(-x // 256) * 256
        # two states a row of the one split: one of each side
        assert K.kamera_attend_shared_workspace_bytes(self.pool.k, self.q, P, len(groups), max(groups), max(prefix),
                                                      0) == align(rows * 2 * d * 4) + align(rows * 2 * 8)

    def slots(self, g, n=None):
        return R.slots_of(self.pre[g].tolist(), self.P, self.prefix[g] if n is None else n, self.pool.n_pages)

    def lists(self):
        out = []
        for s, n in enumerate(self.lens):
            g = int(np.searchsorted(self.starts, s, side="right")) - 1
            out.append(np.concatenate([self.slots(g), R.slots_of(self.own[s].tolist(), self.P, n, self.pool.n_pages)]))
        return out

    def call(self, err=None, **kw):
        return K.kamera_attend_shared(self.pool.k, self.pool.v, self.q, self.P, *self.args, err=err, **kw)


@pytest.mark.parametrize("d,P,G", [(128, 16, 2), (64, 48, 3), (128, 128, 1)])
def test_in_turn_reports_bad_pages(d, P, G):
    """Pages outside the pool in tiles of the first side, of the second, in the first and the
    last tile of a prefix, a whole tile of them, and everywhere."""
    c = InTurn(101, 32, G, d, P, [2, 1, 1, 1], [2049, 1920, 1300, 1153], [50, 0, 33, 7, 64])
    page = lambda token: token // P
    for g, token, bad in ((0, 128 * 3 + 20, -1), (0, 128 * 6 + 100, 2 ** 31 - 1), (0, 2048, -7), (1, 5, -1),
                          (1, 128 * 14 + 1, c.pool.n_pages)):
        c.pre[g, page(token)] = bad
    c.pre[2, page(128 * 5):page(128 * 6 + 127) + 1] = -1      # all of a tile of each side
    c.pre[3, :] = -2
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = c.call(err)
    torch.cuda.synchronize()
    assert int(err.item()) == SLOT
    near(out, lse, rows_ref(c.q, c.pool, c.lists(), d ** -0.5), (d, P, G))


@pytest.mark.parametrize("scale,std", [(-0.09, 1.0), (0.0, 1.0), (0.4, 2.0), (-0.3, 2.0)])
def test_in_turn_of_other_scales(scale, std):
    c = InTurn(102, 32, 2, 128, 16, [1, 2, 1, 1], [1100, 1301, 2176, 128], [20, 0, 33, 5, 40], std)
    out, lse = c.call(scale=scale)
    torch.cuda.synchronize()
    near(out, lse, rows_ref(c.q, c.pool, c.lists(), scale), (scale, std))


@pytest.mark.parametrize("order", [1, -1])
def test_in_turn_of_growing_scores(order):
    """Scores that climb along the prefix (or fall): each side rescales its running output
    again and again, or finds weights that underflow."""
    c = InTurn(103, 32, 2, 128, 32, [1, 1, 2, 1], [1500, 1150, 1281, 1409], [20, 33, 0, 5, 16])
    for g in range(4):
        n = c.prefix[g]
        at = torch.from_numpy(c.slots(g)).to(DEV)
        ramp = torch.linspace(0, 8, n, device=DEV)
        ramp = ramp if order > 0 else ramp.flip(0)
        q = c.q[int(c.starts[g])].float().view(32, 2, 128).sum(1)
        c.pool.k[at] = (c.pool.k[at].float() + ramp[:, None, None] * 0.5 * q).to(torch.bfloat16)
    out, lse = c.call()
    torch.cuda.synchronize()
    near(out, lse, rows_ref(c.q, c.pool, c.lists(), 128 ** -0.5), order)


def test_in_turn_of_infinite_and_nan_scores():
    """Tiles of one side, of the other and of both whose scores are -infinity throughout,
    and a NaN key."""
    c = InTurn(104, 32, 1, 64, 16, [1, 1, 1, 1], [1200, 1290, 1153, 1025], [20, 33, 0, 5])
    c.q.copy_(c.q.abs() + 0.5)
    gone = []
    for g, tiles in ((0, [0, 2, 4]), (1, [1, 3, 5, 9]), (2, [0, 1, 6, 7])):
        t = np.concatenate([np.arange(128 * k, min(128 * k + 128, c.prefix[g])) for k in tiles])
        c.pool.k[torch.from_numpy(c.slots(g)[t]).to(DEV)] = -3e38
        gone.append(t)
    c.pool.k[int(c.slots(3)[700]), 5, 3] = NAN
    out, lse = c.call()
    torch.cuda.synchronize()
    assert bool(torch.isnan(out[3, 5]).all()) and bool(torch.isnan(lse[3, 5]))
    lists = c.lists()
    for g, t in enumerate(gone):
        lists[g] = np.delete(lists[g], t)
    near(out[:3], lse[:3], rows_ref(c.q[:3], c.pool, lists[:3], 64 ** -0.5), "-inf")
    rest = [h for h in range(32) if h != 5]
    refs = rows_ref(c.q[3:], c.pool, lists[3:], 64 ** -0.5)
    near(out[3:][:, rest], lse[3:][:, rest], [refs[h] for h in rest], "beside a NaN")


def test_in_turn_infinite_values():
    c = InTurn(107, 32, 2, 64, 16, [1, 2, 1, 1], [1200, 1290, 1153, 1025], [20, 33, 0, 5, 1])
    for g in range(4):
        at = c.slots(g)
        for j in range(7):
            c.pool.v[int(at[(j * 181 + 37 * g) % c.prefix[g]]), (5 * j + g) % 32, (9 * j) % 64] = INF if j % 2 else -INF
        c.pool.v[int(at[-1]), 3, 63], c.pool.v[int(at[130]), 4, 1], c.pool.v[int(at[300]), 4, 1] = INF, INF, -INF
    out, lse = c.call()
    torch.cuda.synchronize()
    near_with_infinities(out, lse, c.q, c.pool, [[x] * 32 for x in c.lists()], 64 ** -0.5, "in turn")


def test_in_turn_reports_malformed_groups():
    c = InTurn(105, 32, 2, 64, 16, [1, 1, 1, 1], [1200, 1290, 1153, 1025], [20, 33, 0, 5])
    good, _ = c.call()
    for starts, served in (([0, 1, 2, 2, 3], [0, 1]), ([0, 1, 9, 3, 4], [0, 3]), ([0, 1, -7, 3, 4], [0, 3])):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        out, _ = K.kamera_attend_shared(c.pool.k, c.pool.v, c.q, 16, i32(starts), *c.args[1:], err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == DESCRIPTOR, starts
        for s in served:
            assert torch.equal(out[s], good[s]), starts


def test_in_turn_wait_runs_out_then_recovers(monkeypatch):
    """No tile is loaded and every wait gives up after 1 ms: the call returns with
    TIMEOUT, and the next one is right."""
    c = InTurn(106, 32, 2, 128, 16, [1, 1, 1, 1], [1200, 1290, 1153, 1025], [20, 33, 0, 5])
    good, _ = c.call()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    monkeypatch.setenv("KAMERA_WAIT_LIMIT_NS", "1000000")
    monkeypatch.setenv("KAMERA_TEST_WITHHOLD_LOADS", "1")
    c.call(err)
    torch.cuda.synchronize()
    assert int(err.item()) & TIMEOUT
    monkeypatch.delenv("KAMERA_WAIT_LIMIT_NS")
    monkeypatch.delenv("KAMERA_TEST_WITHHOLD_LOADS")
    err.zero_()
    out, _ = c.call(err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(out, good)


# ----------------------------------------------------------------- together --
def test_chunks_relocated_into_the_pages_of_a_table():
    """Chunks reinstated straight into the slots of a shared prefix's page table (the second
    begins inside a page), rows appended behind them, attention over both and over
    selected pages, with no row moved in between."""
    import workloads as W
    from tests import harness as Hn
    spec = W.scaled(W.qwen_recall(), L=1, lens=(130, 75))
    wl = W.make(spec, DEV)
    H, d, P, G, n, pages = spec.H, spec.d, spec.page, 7, 3, 60
    g = torch.Generator(device=DEV).manual_seed(111)
    order = torch.randperm(pages, generator=g, device=DEV).tolist()
    prefix = sum(spec.lens)
    pre = [order.pop() for _ in range(-(-prefix // P))]
    own = [[order.pop(), order.pop()] for _ in range(n)]
    wl.pool_k, wl.pool_v = normal(g, 1, pages * P, H, d), normal(g, 1, pages * P, H, d)
    at = torch.from_numpy(R.slots_of(pre, P, prefix, pages)).to(DEV)
    for c, part in zip(wl.chunks, at.split(list(spec.lens))):
        c.slots = part.to(c.slots.dtype).contiguous()
    before = Hn.snapshot(wl)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    Hn.run_gpu(wl, err=err)
    Hn.check_parity(wl, before, "into pages")
    rope, steps = K.Rope(spec.base, d), P + 3
    for t in range(steps):
        k, v, q = normal(g, n, H, d), normal(g, n, H, d), normal(g, n, H * G, d)
        slot = torch.tensor([own[s][t // P] * P + t % P for s in range(n)], device=DEV)
        turned = K.kamera_append_kv(wl.pool_k, wl.pool_v, k, v, rope, torch.full((n,), prefix + t, device=DEV), slot, q=q,
                                    err=err)
    kk, vv = wl.pool_k[0], wl.pool_v[0]
    lens = i32([steps] * n)
    out, lse = K.kamera_attend_shared(kk, vv, turned, P, i32([0, n]), i32([pre]), i32([prefix]), i32(own), lens, n, prefix,
                                      steps, err=err)
    # the prefix's whole pages and the own ones as one table, and three of them selected
    whole = prefix // P
    table, m = i32([pre[:whole] + own[s] for s in range(n)]), whole * P + steps
    summary = torch.zeros(pages, H, 2, d, dtype=torch.bfloat16, device=DEV)
    ids = i32(pre[:whole] + [p for o in own for p in o[:1]])
    K.kamera_summarize_pages(kk, P, ids, torch.full_like(ids, P), summary, err=err)
    sel = K.kamera_select_pages(turned, summary, P, table, i32([m] * n), m, 5, err=err)
    part, part_lse = K.kamera_attend_selected(kk, vv, turned, P, table, i32([m] * n), sel, m, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    view = Pool.__new__(Pool)
    view.k, view.v, view.H = kk, vv, H
    lists = [np.concatenate([at.cpu().numpy(), R.slots_of(own[s], P, steps, pages)]) for s in range(n)]
    near(out, lse, rows_ref(turned, view, lists, d ** -0.5), "dense")
    chosen = select_ref(turned, summary, table, [m] * n, P, 5, 1, 1)
    assert np.array_equal(sel.cpu().numpy(), chosen)
    qh, refs = R.f64(turned), []
    for s in range(n):
        slots = R.slots_of(table[s].tolist(), P, m, pages)
        for h in range(H):
            idx = torch.from_numpy(np.concatenate([slots[j * P:j * P + P] for j in chosen[s, h]])).to(DEV)
            o, l, a, x = R.attention(qh[s, h * G:h * G + G], R.f64(kk[idx])[:, h], R.f64(vv[idx])[:, h], d ** -0.5)
            refs += [(o[i], l[i], a[i], x[i], len(idx)) for i in range(G)]
    near(part, part_lse, refs, "selected")
