"""Decode attention over the paged pool (kamera_attend_shared,
kamera_attend_selected), page summaries and page selection against their
definitions in 64 bits.

Tolerance of an attention output: its rounding to bf16 (2^-8 relative) plus
the error of the weights times sum_j p_j |V_j|.  A weight's relative error: its
hi + lo split (2^-17), 2^x (2^-21 with the fp32 argument's rounding) and its
score's error, at most (d + 2) 2^-24 of scale sum_i |q_i k_i| (fp32 sums of exact
products) -- in numerator and denominator alike, so twice.  The log-sum-exp: the score's error, the
fp32 sum of n weights (n 2^-24 at the very most) and 2^-21 + 2^-22 |lse| for
2^x, the logarithm and the rounding.  Selected pages are equal as whole numbers,
summaries exact."""
import numpy as np
import pytest
import torch

import position_invariant_kv_chunk_gb300 as K
from tests import paged_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
SLOT, DESCRIPTOR, LEN, TIMEOUT = 1, 4, 8, 32


def normal(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device=DEV) * std).to(torch.bfloat16)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def near(out, lse, refs, what):
    """refs: per (row) tuples (out, lse, mag, smax, n) in 64 bits."""
    d = out.shape[-1]
    ref, rl = np.stack([r[0] for r in refs]), np.array([r[1] for r in refs])
    mag, smax, n = np.stack([r[2] for r in refs]), np.array([r[3] for r in refs]), np.array([r[4] for r in refs])
    got, gl = R.f64(out).reshape(ref.shape), R.f64(lse).reshape(-1)
    score = (d + 2) * 2.0 ** -24 * smax
    tol = R.ulp_half(ref) + (1 + 2.0 ** -8) * 2 * (2.0 ** -17 + 2.0 ** -21 + score)[:, None] * mag
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.abs(got - ref)[bad].max()))
    fin = np.isfinite(rl)
    assert np.array_equal(np.isfinite(gl), fin) and np.all(gl[~fin] == -np.inf), what
    lt = score + n * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -22 * np.abs(rl)
    assert np.all(np.abs(gl[fin] - rl[fin]) <= lt[fin]), (what, float(np.abs(gl[fin] - rl[fin]).max()))


class Pool:
    """A pool of one layer whose unused rows hold NaN, and page tables drawn from it."""

    def __init__(self, seed, n_pages, P, H, d, pad=0, std=1.0, extra_slots=0):
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.P, self.H, self.d, self.n_pages = P, H, d, n_pages
        S = n_pages * P + extra_slots
        wide_k, wide_v = normal(self.g, S, H * d + pad, std=std), normal(self.g, S, H * d + pad)
        self.k = wide_k[:, :H * d].unflatten(1, (H, d))
        self.v = wide_v[:, :H * d].unflatten(1, (H, d))
        self.order = torch.randperm(n_pages, generator=self.g, device=DEV).tolist()
        self.used = torch.zeros(S, dtype=torch.bool, device=DEV)

    def table(self, lens, width=None):
        width = max(-(-max(lens, default=0) // self.P), 1) if width is None else width
        rows = []
        for n in lens:
            pages = [self.order.pop() for _ in range(-(-n // self.P))]
            for j, g in enumerate(pages):
                self.used[g * self.P:g * self.P + min(self.P, n - j * self.P)] = True
            rows.append(pages + [2 ** 31 - 1] * (width - len(pages)))   # past the sequence: never read
        return i32(rows)

    def poison(self):
        self.k[~self.used] = float("nan")
        self.v[~self.used] = float("inf")


def rows_ref(q, pool, slot_lists, scale, rows=None):
    """(out, lse, mag, smax, n) of every (sequence, query head); slot_lists[s] the tokens' slots."""
    n, hq, d = q.shape
    G = hq // pool.H
    qh, out = R.f64(q), []
    for s in range(n):
        keep = slot_lists[s][slot_lists[s] >= 0]
        idx = torch.from_numpy(keep).to(DEV)
        kk, vv = R.f64(pool.k[idx]), R.f64(pool.v[idx])
        for h in range(pool.H):
            o, l, m, x = R.attention(qh[s, h * G:h * G + G], kk[:, h], vv[:, h], scale)
            out += [(o[g], l[g], m[g], x[g], len(keep)) for g in range(G)]
    return out


def shared_case(seed, H, G, d, P, groups, prefix, lens, scale=None, pad=0, std=1.0, extra=0, **kw):
    """groups: sequences of each group; prefix: its length; lens: own lengths.  One
    call against the definition; returns (pool, arguments, out, lse)."""
    n = sum(groups)
    need = sum(-(-x // P) for x in list(prefix) + list(lens)) + 3
    pool = Pool(seed, need, P, H, d, pad, std, extra)
    pre, own = pool.table(prefix, -(-kw.get("max_prefix", max(prefix)) // P) or 1), pool.table(lens)
    pool.poison()
    q = normal(pool.g, n, H * G, d)
    starts = np.concatenate([[0], np.cumsum(groups)])
    args = dict(group_start=i32(starts.tolist()), prefix_pages=pre, prefix_len=i32(list(prefix)), pages=own,
                lens=i32(list(lens)), max_group=max(groups), max_prefix=max(prefix), max_len=max(lens))
    args.update(kw)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = K.kamera_attend_shared(pool.k, pool.v, q, P, scale=scale, err=err, **args)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    slots = []
    for s in range(n):
        g = int(np.searchsorted(starts, s, side="right")) - 1
        slots.append(np.concatenate([R.slots_of(pre[g].tolist(), P, prefix[g], pool.n_pages),
                                     R.slots_of(own[s].tolist(), P, lens[s], pool.n_pages)]))
    near(out, lse, rows_ref(q, pool, slots, d ** -0.5 if scale is None else scale), (seed, H, G, d, P))
    return pool, q, args, out, lse


# ---------------------------------------------------------- shared prefixes --
@pytest.mark.parametrize("prefix", [1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 1000, 2600])
def test_shared_prefix_lengths(prefix):
    shared_case(prefix, H=2, G=7, d=128, P=16, groups=[3], prefix=[prefix], lens=[5, 0, 33])


@pytest.mark.parametrize("P", [16, 32, 48, 64, 80, 128, 256])
def test_shared_page_sizes(P):
    shared_case(P, H=2, G=4, d=64, P=P, groups=[2, 3], prefix=[700, 333], lens=[100, 1, P, P + 1, 2 * P - 1])


@pytest.mark.parametrize("H,G,d", [(1, 1, 64), (1, 1, 128), (3, 16, 128), (2, 9, 64), (32, 1, 128), (1, 8, 128),
                                   (2, 16, 64)])
def test_shared_head_layouts(H, G, d):
    shared_case(H * 100 + G, H=H, G=G, d=d, P=16, groups=[1, 4], prefix=[150, 400], lens=[20, 300, 0, 7, 64])


def test_shared_two_row_tiles_and_ragged_groups():
    """Groups of more rows than one tile holds: full pairs of tiles, a lone tile, a
    few rows; an empty group and a group without a prefix between them."""
    shared_case(11, H=2, G=7, d=128, P=16, groups=[40, 0, 19, 2, 37], prefix=[900, 50, 0, 513, 128],
                lens=[(11 * i) % 70 for i in range(98)])
    shared_case(12, H=1, G=16, d=64, P=32, groups=[50, 3], prefix=[1500, 2100], lens=[(7 * i) % 40 for i in range(53)])


def test_shared_long_prefix_many_splits():
    shared_case(13, H=1, G=8, d=128, P=64, groups=[20], prefix=[30000], lens=[64] * 20)
    shared_case(14, H=1, G=4, d=64, P=16, groups=[2, 1], prefix=[20011, 129], lens=[0, 1, 5000])


@pytest.mark.parametrize("H,G,d,P,groups,prefix,std", [
    (32, 1, 128, 16, [3, 1, 2, 1], [2049, 1100, 128, 0], 1.0),
    (32, 2, 128, 32, [2, 0, 1, 1], [2176, 0, 1793, 1], 3.0),
    (16, 2, 64, 48, [1] * 8, [1500, 1, 1409, 129, 1024, 1025, 640, 127], 1.0)])
def test_shared_long_prefixes_of_few_rows(H, G, d, P, groups, prefix, std):
    """Many (group, KV head) pairs leave each prefix in one piece, and a lone tile of
    rows: its two sides take the tokens' tiles in turn, an odd number or none."""
    shared_case(15 + H + G, H=H, G=G, d=d, P=P, groups=groups, prefix=prefix, std=std,
                lens=[(13 * i) % 50 for i in range(sum(groups))])


def test_shared_peaked_and_growing_scores():
    """Scores up to tens: weights that underflow, and maxima that grow along the
    prefix so that the running output is rescaled."""
    H, G, d, P = 1, 8, 128, 16
    for order in (1, -1):
        pool = Pool(15, 64, P, H, d)
        pre, own = pool.table([700]), pool.table([50, 20])
        q = normal(pool.g, 2, G, d)
        ramp = torch.linspace(0, 6, 700, device=DEV)
        slots = torch.from_numpy(R.slots_of(pre[0].tolist(), P, 700, 64)).to(DEV)
        ramp = ramp if order > 0 else ramp.flip(0)
        pool.k[slots] = (pool.k[slots].float() + ramp[:, None, None] * q[0, 0].float()).to(torch.bfloat16)
        pool.poison()
        out, lse = K.kamera_attend_shared(pool.k, pool.v, q, P, i32([0, 2]), pre, i32([700]), own, i32([50, 20]), 2,
                                          700, 50)
        torch.cuda.synchronize()
        lists = [np.concatenate([slots.cpu().numpy(), R.slots_of(own[s].tolist(), P, n, 64)])
                 for s, n in ((0, 50), (1, 20))]
        near(out, lse, rows_ref(q, pool, lists, d ** -0.5), order)


@pytest.mark.parametrize("scale", [0.0, -0.09, 0.5])
def test_shared_other_scales(scale):
    shared_case(16, H=1, G=3, d=64, P=16, groups=[2], prefix=[300], lens=[40, 3], scale=scale)


def test_shared_strided_pool_with_a_part_page_at_its_end():
    shared_case(17, H=2, G=4, d=64, P=32, groups=[3], prefix=[200], lens=[10, 70, 0], pad=40, extra=17)


def test_shared_without_prefix_or_own_tokens():
    _, _, _, out, lse = shared_case(18, H=2, G=4, d=128, P=16, groups=[1, 1, 1], prefix=[0, 0, 0], lens=[0, 700, 16],
                                    max_prefix=512)
    assert not bool(out[0].any()) and bool((lse[0] == -float("inf")).all())
    pool = Pool(19, 40, 16, 2, 64)
    table = pool.table([300, 0])
    pool.poison()
    q = normal(pool.g, 2, 6, 64)
    # own tokens alone
    out, lse = K.kamera_attend_shared(pool.k, pool.v, q, 16, None, None, None, table, i32([300, 0]), 0, 0, 300)
    # the same as a prefix alone, each sequence its own group
    out2, lse2 = K.kamera_attend_shared(pool.k, pool.v, q, 16, i32([0, 1, 2]), table, i32([300, 0]), None, None, 1,
                                        300, 0)
    torch.cuda.synchronize()
    lists = [R.slots_of(table[0].tolist(), 16, 300, 40), np.zeros(0, dtype=np.int64)]
    ref = rows_ref(q, pool, lists, 64 ** -0.5)
    near(out, lse, ref, "own alone")
    near(out2, lse2, ref, "prefix alone")
    # no token anywhere
    out, lse = K.kamera_attend_shared(pool.k, pool.v, q, 16, None, None, None, None, None, 0, 0, 0)
    torch.cuda.synchronize()
    assert not bool(out.any()) and bool((lse == -float("inf")).all())


def test_shared_reports_bad_pages_and_lengths():
    """A page outside the pool leaves its tokens out; a length past its bound reads as empty."""
    H, G, d, P = 2, 7, 128, 16
    pool = Pool(20, 60, P, H, d)
    pre, own = pool.table([400]), pool.table([50, 33])
    pool.poison()
    q = normal(pool.g, 2, H * G, d)
    pre[0, 3], pre[0, 24], own[0, 1], own[1, 2] = -5, 60, 2 ** 31 - 1, -1
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = K.kamera_attend_shared(pool.k, pool.v, q, P, i32([0, 2]), pre, i32([400]), own, i32([50, 33]), 2, 400,
                                      50, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == SLOT
    lists = [np.concatenate([R.slots_of(pre[0].tolist(), P, 400, 60), R.slots_of(own[s].tolist(), P, n, 60)])
             for s, n in ((0, 50), (1, 33))]
    near(out, lse, rows_ref(q, pool, lists, d ** -0.5), "bad pages")
    err.zero_()
    out, lse = K.kamera_attend_shared(pool.k, pool.v, q, P, i32([0, 2]), pre, i32([400]), own, i32([49, -1]), 2, 399,
                                      48, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == LEN
    assert not bool(out.any()) and bool((lse == -float("inf")).all())


@pytest.mark.parametrize("G", [4, 16])
def test_shared_reports_malformed_groups(G):
    """Group starts out of order or past the batch, and a sequence in no group: the
    call reports them, reads nothing out of range and serves the other sequences."""
    pool = Pool(21, 40, 16, 1, 64)
    pre, own = pool.table([100, 90, 80]), pool.table([20, 20, 20])
    pool.poison()
    q = normal(pool.g, 3, G, 64)
    good, _ = K.kamera_attend_shared(pool.k, pool.v, q, 16, i32([0, 1, 2, 3]), pre, i32([100, 90, 80]), own,
                                     i32([20, 20, 20]), 1, 100, 20)
    for starts, served in (([0, 1, 1, 2], [0]), ([0, 1, 9, 3], [0]), ([0, 1, -7, 3], [0]), ([-1, 1, 2, 3], [1, 2])):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        out, _ = K.kamera_attend_shared(pool.k, pool.v, q, 16, i32(starts), pre, i32([100, 90, 80]), own,
                                        i32([20, 20, 20]), 1, 100, 20, err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == DESCRIPTOR, starts
        for s in served:
            assert torch.equal(out[s], good[s]), starts


def test_shared_infinite_and_nan_scores():
    """Keys that make scores -infinity carry no weight; a NaN key makes its sequence's rows NaN."""
    H, G, d, P = 1, 4, 64, 16
    pool = Pool(22, 60, P, H, d)
    pre, own = pool.table([300]), pool.table([40, 200, 30])
    pool.poison()
    q = normal(pool.g, 3, G, d).abs() + 0.5
    down = torch.from_numpy(R.slots_of(pre[0].tolist(), P, 300, 60)[:140]).to(DEV)
    pool.k[down] = -3e38                                                 # the first tile and more: -infinity
    nan = int(R.slots_of(own[1].tolist(), P, 200, 60)[150])
    pool.k[nan, 0, 3] = float("nan")
    out, lse = K.kamera_attend_shared(pool.k, pool.v, q, P, i32([0, 3]), pre, i32([300]), own, i32([40, 200, 30]), 3,
                                      300, 200)
    torch.cuda.synchronize()
    assert bool(torch.isnan(out[1]).all()) and bool(torch.isnan(lse[1]).all())
    keep = [0, 2]
    lists = [np.concatenate([R.slots_of(pre[0].tolist(), P, 300, 60)[140:], R.slots_of(own[s].tolist(), P, n, 60)])
             for s, n in ((0, 40), (2, 30))]
    near(out[keep], lse[keep], rows_ref(q[keep], pool, lists, d ** -0.5), "-inf")


def test_shared_past_32_bit_offsets():
    """Pages whose element offsets pass 2^32 in a tall pool."""
    H, G, d, P, S = 8, 2, 128, 16, (1 << 22) + 64
    pool = Pool.__new__(Pool)
    pool.g = torch.Generator(device=DEV).manual_seed(23)
    pool.k = torch.zeros(S, H, d, dtype=torch.bfloat16, device=DEV)
    pool.v = torch.zeros(S, H, d, dtype=torch.bfloat16, device=DEV)
    pool.P, pool.H, pool.d, pool.n_pages = P, H, d, S // P
    last = S // P - 1
    pages = [last, 5, last - 9, S // P // 2, last - 1, 0, last - 2, 17, last - 3, 3]
    rows = torch.cat([torch.arange(g * P, g * P + P, device=DEV) for g in pages])
    pool.k[rows], pool.v[rows] = normal(pool.g, 160, H, d), normal(pool.g, 160, H, d)
    q = normal(pool.g, 2, H * G, d)
    pre, own = i32([pages[:7]]), i32([pages[7:], pages[7:]])
    out, lse = K.kamera_attend_shared(pool.k, pool.v, q, P, i32([0, 2]), pre, i32([110]), own, i32([48, 20]), 2, 110,
                                      48)
    torch.cuda.synchronize()
    lists = [np.concatenate([R.slots_of(pages[:7], P, 110, pool.n_pages), R.slots_of(pages[7:], P, n, pool.n_pages)])
             for n in (48, 20)]
    near(out, lse, rows_ref(q, pool, lists, d ** -0.5), "tall pool")


def test_shared_captured_graphs_and_streams():
    """Two captured calls replayed together on two streams, a call on a side stream
    and a plain one agree bit for bit (each graph has a workspace of its own)."""
    H, G, d, P = 2, 7, 128, 16
    pool = Pool(24, 400, P, H, d)
    pre, own = pool.table([2000]), pool.table([700, 5, 300, 64])
    pool.poison()
    qs = [normal(pool.g, 4, H * G, d) for _ in range(2)]
    args = (P, i32([0, 4]), pre, i32([2000]), own, i32([700, 5, 300, 64]), 4, 2000, 700)
    plain = [K.kamera_attend_shared(pool.k, pool.v, q, *args) for q in qs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = K.kamera_attend_shared(pool.k, pool.v, qs[0], *args, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(other[0], plain[0][0]) and torch.equal(other[1], plain[0][1])
    graphs, outs = [], []
    for q in qs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(K.kamera_attend_shared(pool.k, pool.v, q, *args))
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for o in outs:
            o[0].zero_()
        torch.cuda.synchronize()
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for o, p in zip(outs, plain):
            assert torch.equal(o[0], p[0]) and torch.equal(o[1], p[1])


@pytest.mark.parametrize("what", ["prefix", "own"])
def test_shared_wait_runs_out_then_recovers(what, monkeypatch):
    """No tile is loaded and every wait gives up after 1 ms: the call returns with
    TIMEOUT, and the next one is right (tensor memory was freed)."""
    pool = Pool(25, 100, 16, 2, 128)
    pre = pool.table([600 if what == "prefix" else 0], 38)
    own = pool.table([200 if what == "own" else 0] * 2, 13)
    pool.poison()
    q = normal(pool.g, 2, 14, 128)
    args = (16, i32([0, 2]), pre, i32([600 if what == "prefix" else 0]), own, i32([200 if what == "own" else 0] * 2),
            2, 600, 200)
    good, _ = K.kamera_attend_shared(pool.k, pool.v, q, *args)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    monkeypatch.setenv("KAMERA_WAIT_LIMIT_NS", "1000000")
    monkeypatch.setenv("KAMERA_TEST_WITHHOLD_LOADS", "1")
    K.kamera_attend_shared(pool.k, pool.v, q, *args, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) & TIMEOUT
    monkeypatch.delenv("KAMERA_WAIT_LIMIT_NS")
    monkeypatch.delenv("KAMERA_TEST_WITHHOLD_LOADS")
    err.zero_()
    out, _ = K.kamera_attend_shared(pool.k, pool.v, q, *args, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and torch.equal(out, good)


# ---------------------------------------------------------------- summaries --
@pytest.mark.parametrize("P,H,d,n", [(16, 4, 128, 37), (48, 2, 64, 5), (128, 1, 8, 3), (64, 3, 80, 1),
                                     (16, 8, 128, 700)])
def test_summaries_are_exact(P, H, d, n):
    g = torch.Generator(device=DEV).manual_seed(n)
    N = n + 5
    wide = normal(g, N * P + 7, H * d + 16)
    pool = wide[:, :H * d].unflatten(1, (H, d))
    ids = torch.randperm(N, generator=g, device=DEV)[:n].to(torch.int32)
    tokens = torch.randint(1, P + 1, (n,), generator=g, device=DEV, dtype=torch.int32)
    tokens[0] = 1
    if n > 2:
        tokens[1], tokens[2] = P, 0
    if n > 3:
        pool[int(ids[3]) * P, 0, 5] = float("nan")
    summary = normal(g, N, H, 2, d)
    ref = summary.clone()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    K.kamera_summarize_pages(pool, P, ids, tokens, summary, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for page, c in zip(ids.tolist(), tokens.tolist()):
        if c:
            rows = pool[page * P:page * P + c]
            ref[page, :, 0], ref[page, :, 1] = rows.amin(0), rows.amax(0)
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(summary), nan)
    assert torch.equal(summary.nan_to_num(), ref.nan_to_num())
    if n > 3:
        assert int(nan.sum()) == 2


def test_summaries_report_bad_entries():
    pool = torch.randn(64, 2, 64, device=DEV).to(torch.bfloat16)
    summary = torch.zeros(4, 2, 2, 64, dtype=torch.bfloat16, device=DEV)
    for page, c, bit in ((4, 3, SLOT), (-1, 3, SLOT), (1, 17, LEN), (1, -1, LEN)):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        K.kamera_summarize_pages(pool, 16, i32([page, 2]), i32([c, 16]), summary.zero_(), err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == bit
        assert torch.equal(summary[2, :, 1], pool[32:48].amax(0))
        summary[2] = 0
        assert not bool(summary.any())


# ----------------------------------------------------------------- selection --
def select_ref(q, summary, pages, lens, P, k, nf, nl):
    n, hq, d = q.shape
    H = summary.shape[1]
    G = hq // H
    qh, sh, out = R.f64(q), R.f64(summary), []
    for s in range(n):
        count = -(-lens[s] // P)
        box = sh[pages[s, :count].long().cpu().numpy()]
        for h in range(H):
            out.append(R.select(R.page_scores(qh[s, h * G:h * G + G], box[:, h, 0], box[:, h, 1]), k, nf, nl))
    return np.array(out, dtype=np.int64).reshape(n, H, k)


def boxes(g, N, H, d):
    a, b = normal(g, N, H, d), normal(g, N, H, d)
    return torch.stack([torch.minimum(a, b), torch.maximum(a, b)], dim=2).contiguous()


@pytest.mark.parametrize("H,G,d,P,k,nf,nl", [(4, 7, 128, 16, 64, 1, 1), (2, 1, 64, 64, 2, 1, 1), (1, 16, 128, 16, 5, 0, 0),
                                             (2, 8, 64, 48, 33, 2, 3), (1, 4, 128, 32, 4, 2, 2), (3, 9, 64, 16, 1, 0, 1)])
def test_selection_is_the_exact_one(H, G, d, P, k, nf, nl):
    g = torch.Generator(device=DEV).manual_seed(H * G + k)
    lens = [1, P, P + 1, k * P, k * P + 1, 0, 3000, 9000]
    width = -(-max(lens) // P)
    N = width + 30
    summary = boxes(g, N, H, d)
    pages = torch.stack([torch.randperm(N, generator=g, device=DEV)[:width] for _ in lens]).to(torch.int32)
    q = normal(g, len(lens), H * G, d)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = K.kamera_select_pages(q, summary, P, pages, i32(lens), max(lens), k, nf, nl, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert np.array_equal(got.cpu().numpy(), select_ref(q, summary, pages, lens, P, k, nf, nl))


@pytest.mark.parametrize("n,pages_of_one", [(1, 2048), (1, 2049), (3, 700), (10, 200), (38, 97), (39, 97), (50, 130)])
def test_selection_of_few_and_many_rows(n, pages_of_one):
    """Rows that share a launch with their scores, by one to eight CTAs each, and rows
    that are too many or too long for it; ragged, some with every page taken."""
    H, G, d, P, k = 4, 3, 64, 16, 9
    g = torch.Generator(device=DEV).manual_seed(n)
    lens = [(pages_of_one if s == n - 1 else (s * 37) % pages_of_one) * P - (s % 5 if s else 0) for s in range(n)]
    lens = [max(x, 0) for x in lens]
    N = pages_of_one + 5
    summary = boxes(g, N, H, d)
    pages = torch.stack([torch.randperm(N, generator=g, device=DEV)[:pages_of_one] for _ in lens]).to(torch.int32)
    q = normal(g, n, H * G, d)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    ref = select_ref(q, summary, pages, lens, P, k, 1, 1)
    for _ in range(3):
        got = K.kamera_select_pages(q, summary, P, pages, i32(lens), pages_of_one * P, k, 1, 1, err=err)
        assert np.array_equal(got.cpu().numpy(), ref)
    assert int(err.item()) == 0


@pytest.mark.parametrize("N", [2000, 5000])
def test_selection_among_many_nearly_equal_pages(N):
    """More pages near the border than are ranked at once: boxes that differ in one
    channel by the least bf16 steps there are, and equal ones among them."""
    H, G, d, P, k = 1, 2, 128, 16, 700
    g = torch.Generator(device=DEV).manual_seed(N)
    one = normal(g, 1, H, 1, d).expand(N, H, 2, d).contiguous()
    steps = torch.randint(0, 500, (N,), generator=g, device=DEV)
    one[:, 0, :, 3] = (steps.float() * 2.0 ** -30)[:, None].to(torch.bfloat16)
    pages = torch.randperm(N, generator=g, device=DEV).to(torch.int32)[None]
    q = normal(g, 1, H * G, d)
    q[:, :, 3] = 1.0
    got = K.kamera_select_pages(q, one, P, pages, i32([N * P]), N * P, k, 1, 1)
    assert np.array_equal(got.cpu().numpy(), select_ref(q, one, pages, [N * P], P, k, 1, 1))


def test_selection_ties_go_to_the_lower_page():
    """Few distinct boxes over many pages, and boxes all alike: equal scores by the
    hundred, more than are ranked by comparison, at every level of the search."""
    g = torch.Generator(device=DEV).manual_seed(31)
    H, G, d, P, width = 2, 4, 64, 16, 5000
    lens = [width * P, width * P - 3, 1700 * P, 40 * P]
    kinds = boxes(g, 3, H, d)
    pages = torch.stack([torch.randperm(width, generator=g, device=DEV) for _ in lens]).to(torch.int32)
    for few in (1, 3):
        pick = torch.randint(0, few, (width,), generator=g, device=DEV)
        summary = kinds[pick].contiguous()
        for k in (2, 100, 1666, 1700, 3500):
            q = normal(g, len(lens), H * G, d)
            got = K.kamera_select_pages(q, summary, P, pages, i32(lens), max(lens), k)
            torch.cuda.synchronize()
            assert np.array_equal(got.cpu().numpy(), select_ref(q, summary, pages, lens, P, k, 1, 1)), (few, k)


def test_selection_close_scores():
    """Scores that differ by one part in 2^30 and less of their terms: fp32 sums would
    not tell them apart, the pairs of floats do."""
    H, G, d, P, n = 1, 1, 128, 16, 400
    g = torch.Generator(device=DEV).manual_seed(32)
    base = normal(g, d)
    box = base[None].repeat(n, 1)
    box[:, 7] = 2.0 ** -31 * (torch.randperm(n, generator=g, device=DEV) % 251).to(torch.bfloat16)   # 8 bits: exact
    summary = torch.stack([box, box], dim=1)[:, None].contiguous()
    q = normal(g, 1, 1, d)
    q[0, 0, 7] = 1.0
    pages = torch.randperm(n, generator=g, device=DEV)[None].to(torch.int32)
    got = K.kamera_select_pages(q, summary, P, pages, i32([n * P]), n * P, 100)
    torch.cuda.synchronize()
    lo = [[float(x) for x in row] for row in box.double().cpu()]
    # the common part drops out of the order: what is left is the exact last term
    score = np.array([lo[j][7] for j in pages[0].tolist()])
    assert got[0, 0].tolist() == R.select(score, 100, 1, 1)


def test_selection_infinities_nan_and_bad_pages():
    """Scores that are not finite come first, a page outside the summary last."""
    H, G, d, P, n = 1, 1, 64, 16, 50
    g = torch.Generator(device=DEV).manual_seed(33)
    summary = boxes(g, n, H, d)
    q = normal(g, 1, 1, d).abs() + 0.25
    summary[11, 0, 1, 3] = float("inf")
    summary[30, 0, 1, 9] = float("nan")
    summary[20, 0, :, 5] = -float("inf")
    pages = i32([list(range(n))])
    pages[0, 40] = n
    pages[0, 41] = -1
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    for k, inside, outside in ((4, [11, 20], [30]), (5, [11, 20, 30], []), (48, [11, 20, 30], [40, 41]),
                               (49, [11, 20, 30, 40], [41])):
        got = K.kamera_select_pages(q, summary, P, pages, i32([n * P]), n * P, k, err=err)
        torch.cuda.synchronize()
        row = got[0, 0].tolist()
        assert row == sorted(row) and len(set(row)) == k and 0 in row and n - 1 in row
        assert all(j in row for j in inside), (k, row)
        assert not any(j in row for j in outside), (k, row)
    assert int(err.item()) == SLOT


def test_selection_reads_no_forced_summary_and_long_rows():
    """NaN summaries of the first and last pages change nothing; a row too long for
    the keys to stay in shared memory is chosen from alike."""
    H, G, d, P, k = 1, 2, 64, 16, 70
    g = torch.Generator(device=DEV).manual_seed(34)
    width = 13000
    summary = boxes(g, width, H, d)
    pages = torch.randperm(width, generator=g, device=DEV)[None].to(torch.int32)
    q = normal(g, 1, H * G, d)
    lens = [width * P - 5]
    ref = select_ref(q, summary, pages, lens, P, k, 2, 2)
    for j in (0, 1, width - 2, width - 1):
        summary[pages[0, j].long()] = float("nan")
    got = K.kamera_select_pages(q, summary, P, pages, i32(lens), width * P, k, 2, 2)
    torch.cuda.synchronize()
    assert np.array_equal(got.cpu().numpy(), ref)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = K.kamera_select_pages(q, summary, P, pages, i32([width * P + 1]), width * P, k, 2, 2, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == LEN and bool((got == -1).all())


# -------------------------------------------------------- selected attention --
@pytest.mark.parametrize("H,G,d,P", [(4, 7, 128, 16), (2, 16, 64, 48), (1, 1, 128, 64), (2, 9, 128, 32)])
def test_selected_attention_matches_definition(H, G, d, P):
    lens = [1, P, P + 3, 20 * P, 20 * P - 7, 0]
    pool = Pool(H + G, sum(-(-x // P) for x in lens) + 2, P, H, d)
    pages = pool.table(lens)
    pool.poison()
    q = normal(pool.g, len(lens), H * G, d)
    k = 9
    sel = torch.full((len(lens), H, k), -1, dtype=torch.int32, device=DEV)
    rng = np.random.default_rng(5)
    for s, n in enumerate(lens):
        count = -(-n // P)
        for h in range(H):
            take = rng.permutation(count)[:rng.integers(0, k + 1)]
            if s == 4:
                take = np.unique(np.append(take[:k - 1], count - 1))      # the part page at the end
            where = rng.permutation(k)[:len(take)]                        # -1 between, any order
            for i, j in zip(where, take):
                sel[s, h, i] = int(j)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, lse = K.kamera_attend_selected(pool.k, pool.v, q, P, pages, i32(lens), sel, max(lens), err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    qh, refs = R.f64(q), []
    for s, n in enumerate(lens):
        slots = R.slots_of(pages[s].tolist(), P, n, pool.n_pages)
        for h in range(H):
            t = [x for j in sel[s, h].tolist() if j >= 0 for x in range(j * P, min(n, j * P + P))]
            idx = torch.from_numpy(slots[t] if t else np.zeros(0, dtype=np.int64)).to(DEV)
            o, l, m, x = R.attention(qh[s, h * G:h * G + G], R.f64(pool.k[idx])[:, h], R.f64(pool.v[idx])[:, h], d ** -0.5)
            refs += [(o[g], l[g], m[g], x[g], len(t)) for g in range(G)]
    near(out, lse, refs, (H, G, d, P))
    sel[3, 0, 0] = 20                                                     # past the sequence: reported, left out
    K.kamera_attend_selected(pool.k, pool.v, q, P, pages, i32(lens), sel, max(lens), err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == SLOT


def test_selected_nothing_and_given_buffers():
    """No page selected (an empty selection, or -1 throughout): zeros and -infinity; the
    caller's out, lse and workspace are used, and lse False leaves it out."""
    H, G, d, P = 2, 4, 64, 16
    lens = [100, 37]
    pool = Pool(42, 30, P, H, d)
    pages = pool.table(lens)
    pool.poison()
    q = normal(pool.g, 2, H * G, d)
    for k in (0, 3):
        sel = torch.full((2, H, k), -1, dtype=torch.int32, device=DEV)
        out, lse = K.kamera_attend_selected(pool.k, pool.v, q, P, pages, i32(lens), sel, 100)
        torch.cuda.synchronize()
        assert not bool(out.any()) and bool((lse == -float("inf")).all()), k
    args = (pool.k, pool.v, q, P, i32([0, 2]), pages[:1].contiguous(), i32([90]), pages, i32(lens), 2, 90, 100)
    out, lse = K.kamera_attend_shared(*args)
    mine = torch.empty_like(out), torch.empty_like(lse)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)
    got = K.kamera_attend_shared(*args, out=mine[0], lse=mine[1], workspace=ws)
    none = K.kamera_attend_shared(*args, lse=False)
    torch.cuda.synchronize()
    assert got[0] is mine[0] and got[1] is mine[1] and none[1] is None
    assert torch.equal(out, mine[0]) and torch.equal(lse, mine[1]) and torch.equal(out, none[0])
    with pytest.raises(K.KameraError):
        K.kamera_attend_shared(*args, workspace=ws[:64])


@pytest.mark.parametrize("lens", [[4000], [1500, 1, 0], [700] * 5])
def test_own_pages_by_cluster_and_by_merge(lens):
    """Sequences without a prefix whose splits join in a cluster, and the same beside a
    prefix of no token, where they join through the workspace."""
    H, G, d, P = 2, 7, 128, 16
    n = len(lens)
    pool = Pool(43, sum(-(-x // P) for x in lens) + 4, P, H, d)
    table = pool.table(lens)
    pool.poison()
    q = normal(pool.g, n, H * G, d)
    a = K.kamera_attend_shared(pool.k, pool.v, q, P, None, None, None, table, i32(lens), 0, 0, max(lens))
    b = K.kamera_attend_shared(pool.k, pool.v, q, P, i32([0, n]), table[:1].contiguous(), i32([0]), table, i32(lens), n,
                               16, max(lens))
    torch.cuda.synchronize()
    refs = rows_ref(q, pool, [R.slots_of(table[s].tolist(), P, x, pool.n_pages) for s, x in enumerate(lens)], d ** -0.5)
    near(*a, refs, "cluster")
    near(*b, refs, "merge")


def test_calls_in_a_row_see_each_others_writes():
    """Append, attend, append, summarise, select, attend without a wait between: each
    call starts while the one before ends, and must still see what it wrote."""
    H, G, d, P, n = 4, 7, 128, 16, 6
    pool = Pool(44, 500, P, H, d)
    lens0 = [700, 33, 1200, 16, 5, 900]
    table = pool.table([x + 40 for x in lens0])
    k4, v4 = pool.k.unsqueeze(0), pool.v.unsqueeze(0)
    summary = torch.zeros(500, H, 2, d, dtype=torch.bfloat16, device=DEV)
    q = normal(pool.g, n, H * G, d)
    rows = [(normal(pool.g, n, H, d), normal(pool.g, n, H, d)) for _ in range(24)]
    rope = K.Rope(1e4, d)
    slots = [torch.tensor([int(table[s, (lens0[s] + t) // P]) * P + (lens0[s] + t) % P for s in range(n)], device=DEV)
             for t in range(24)]
    pos = [torch.tensor([lens0[s] + t for s in range(n)], device=DEV) for t in range(24)]
    lens = [i32([x + t + 1 for x in lens0]) for t in range(24)]
    ids = i32([int(table[s, j]) for s in range(n) for j in range(-(-(lens0[s] + 24) // P))])
    full = torch.full_like(ids, P)
    start, before = torch.clone(pool.k), torch.clone(pool.v)

    def steps(wait):
        pool.k.copy_(start)
        pool.v.copy_(before)
        got = []
        for t in range(24):
            turned = K.kamera_append_kv(k4, v4, *rows[t], rope, pos[t], slots[t], q=q)
            wait()
            got += K.kamera_attend_shared(pool.k, pool.v, turned, P, i32([0, 3, n]), table[:2].contiguous(),
                                          i32([600, 20]), table, lens[t], 3, 600, 1240)
            wait()
            K.kamera_summarize_pages(pool.k, P, ids, full, summary)
            wait()
            sel = K.kamera_select_pages(turned, summary, P, table, lens[t], 1240, 9)
            wait()
            got += [sel, *K.kamera_attend_selected(pool.k, pool.v, turned, P, table, lens[t], sel, 1240)]
            wait()
        return got

    alone = steps(torch.cuda.synchronize)
    for _ in range(5):
        together = steps(lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, together))


def test_selecting_every_page_is_dense_attention():
    """Selecting all pages gives what attention over the whole sequence gives."""
    H, G, d, P = 2, 4, 64, 16
    lens = [500, 37, 0, 16]
    pool = Pool(41, 60, P, H, d)
    pages = pool.table(lens)
    pool.poison()
    q = normal(pool.g, 4, H * G, d)
    summary = torch.zeros(60, H, 2, d, dtype=torch.bfloat16, device=DEV)
    sel = K.kamera_select_pages(q, summary, P, pages, i32(lens), 500, 32)
    out, lse = K.kamera_attend_selected(pool.k, pool.v, q, P, pages, i32(lens), sel, 500)
    torch.cuda.synchronize()
    lists = [R.slots_of(pages[s].tolist(), P, n, 60) for s, n in enumerate(lens)]
    near(out, lse, rows_ref(q, pool, lists, d ** -0.5), "all pages")


# ---------------------------------------------------------------- together --
def test_decode_steps_together():
    """Reused chunks relocated into the pool as a shared prefix, then decode steps:
    append the new token, attend over prefix and own pages, summarise the pages,
    select and attend over the selection -- each against 64-bit arithmetic on the
    rows that the pool holds."""
    import workloads as W
    from tests import harness as Hn
    spec = W.scaled(W.qwen_recall(), L=1, lens=(130, 75))
    wl = W.make(spec, DEV)
    Hn.run_gpu(wl)                                          # the prefix: two relocated chunks in wl's pool
    torch.cuda.synchronize()
    H, d, P, G, n = spec.H, spec.d, spec.page, 7, 3
    slots = torch.cat([c.slots for c in wl.chunks]).cpu().numpy()
    g = torch.Generator(device=DEV).manual_seed(51)
    used = set((slots // P).tolist())
    total = wl.pool_k.shape[1] // P
    more = 40
    pool_k = torch.cat([wl.pool_k, normal(g, 1, more * P, H, d)], dim=1).contiguous()
    pool_v = torch.cat([wl.pool_v, normal(g, 1, more * P, H, d)], dim=1).contiguous()
    # a prefix by pages: the chunks' rows copied behind one another into whole pages
    prefix = len(slots)
    pre_pages = list(range(total, total + -(-prefix // P)))
    at = torch.tensor([pre_pages[t // P] * P + t % P for t in range(prefix)], device=DEV)
    src = torch.from_numpy(slots).to(DEV)
    pool_k[0, at], pool_v[0, at] = pool_k[0, src], pool_v[0, src]
    free = [p for p in range(total + more - 1, -1, -1) if p not in used and p not in pre_pages]
    own = [[free.pop(0), free.pop(0)] for _ in range(n)]
    table = i32(own)
    rope = K.Rope(spec.base, d)
    Hq = H * G
    steps = P + 3                                           # into the second page
    for t in range(steps):
        rows = normal(g, n, (Hq + 2 * H) * d)
        q = rows[:, :Hq * d].unflatten(1, (Hq, d))
        k = rows[:, Hq * d:(Hq + H) * d].unflatten(1, (H, d))
        v = rows[:, (Hq + H) * d:].unflatten(1, (H, d))
        pos = torch.full((n,), prefix + t, device=DEV)
        slot = torch.tensor([own[s][t // P] * P + t % P for s in range(n)], device=DEV)
        turned = K.kamera_append_kv(pool_k, pool_v, k, v, rope, pos, slot, q=q)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    lens = i32([steps] * n)
    out, lse = K.kamera_attend_shared(pool_k[0], pool_v[0], turned, P, i32([0, n]), i32([pre_pages]), i32([prefix]),
                                      table, lens, n, prefix, steps, err=err)
    m = (prefix // P) * P                                   # a page table holds whole pages: the prefix's part page is left out
    sparse_pages = i32([pre_pages[:prefix // P] + own[s] for s in range(n)])
    summary = torch.zeros(total + more, H, 2, d, dtype=torch.bfloat16, device=DEV)
    ids = i32(pre_pages[:prefix // P] + [p for o in own for p in o[:1]])
    K.kamera_summarize_pages(pool_k[0], P, ids, torch.full_like(ids, P), summary, err=err)
    sel = K.kamera_select_pages(turned, summary, P, sparse_pages, i32([m + steps] * n), m + steps, 6, err=err)
    out2, lse2 = K.kamera_attend_selected(pool_k[0], pool_v[0], turned, P, sparse_pages, i32([m + steps] * n), sel,
                                          m + steps, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    inv = spec.base ** (-2.0 * np.arange(d // 2) / d)
    ref = R.turned(R.f64(q), pos.cpu().numpy(), inv, 0, False)
    assert np.all(np.abs(R.f64(turned) - ref) <= R.ulp_half(ref) + 2.0 ** -20 * (1 + 2.0 ** -8)
                  * R.turn_scale(R.f64(q), d // 2, 0, False))

    class P_:
        pass
    view = P_()
    view.k, view.v, view.H = pool_k[0], pool_v[0], H
    lists = [np.concatenate([at.cpu().numpy(), R.slots_of(own[s], P, steps, total + more)]) for s in range(n)]
    near(out, lse, rows_ref(turned, view, lists, d ** -0.5), "dense step")
    chosen = select_ref(turned, summary, sparse_pages, [m + steps] * n, P, 6, 1, 1)
    assert np.array_equal(sel.cpu().numpy(), chosen)
    qh, refs = R.f64(turned), []
    for s in range(n):
        slots_s = R.slots_of(sparse_pages[s].tolist(), P, m + steps, total + more)
        for h in range(H):
            t = [x for j in chosen[s, h] if j >= 0 for x in range(j * P, min(m + steps, j * P + P))]
            idx = torch.from_numpy(slots_s[t]).to(DEV)
            o, l, mg, x = R.attention(qh[s, h * G:h * G + G], R.f64(pool_k[0][idx])[:, h], R.f64(pool_v[0][idx])[:, h],
                                      d ** -0.5)
            refs += [(o[i], l[i], mg[i], x[i], len(t)) for i in range(G)]
    near(out2, lse2, refs, "sparse step")
