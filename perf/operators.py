"""Measured cases of the decode-step operators over the paged pool: appending new rows with their
rotation, attention of a batch that shares a prefix, and attention over selected pages.

Each case names its operator in ``op``; ``prepare`` draws what a serving loop holds before the call,
``run`` makes one pass (the plain form in elementary torch operations, or the library's entry points
when ``own`` is set), ``exact`` states the same result from the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
QWEN = dict(H=4, G=7, d=128, base=1e6)     # Qwen2.5-VL-7B shaped heads: 28 query heads on 4 KV heads
MHA = dict(H=32, G=1, d=128, base=1e4)     # the MHA workload's 32 heads
TINY = dict(H=2, G=4, d=64, base=1e4)      # 2 KV heads of 64


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one decode step of 64 sequences: one new token each, queries rotated on the way (latency)
        dict(name="append_step", op="append", tokens=64, page=16, q=True, **QWEN),
        # the rows of eight 1296-token frames entering the pool at prefill
        dict(name="append_frames", op="append", tokens=10368, page=16, q=True, **QWEN),
        # a DeepSeek-V2-Lite shaped prompt: latent row copied, k_rope and 16 rope queries rotated
        dict(name="append_mla", op="append_mla", tokens=16381, page=64, lora=512, rope=64, Hq=16, base=1e4),
        # four short questions about one frame (latency)
        dict(name="shared_one_frame", op="shared", seqs=4, groups=1, prefix=1296, tail=37, page=16, **QWEN),
        # 32 questions about the same eight frames
        dict(name="shared_frames", op="shared", seqs=32, groups=1, prefix=10368, tail=509, page=16, **QWEN),
        # four documents, 16 readers each, MHA heads (no head shares a key: only the batch does)
        dict(name="shared_mha", op="shared", seqs=64, groups=4, prefix=4099, tail=256, page=64, **MHA),
        # a long video read by 64 sequences: the largest
        dict(name="shared_long", op="shared", seqs=64, groups=1, prefix=98304, tail=1024, page=16, **QWEN),
        # page summaries of a whole 131072-token window, written once when it fills
        dict(name="summary_window", op="summary", pages=8192, page=16, **QWEN),
        # one user, 32768 tokens, 64 pages of 16 chosen per step (latency)
        dict(name="sparse_one", op="sparse", seqs=1, context=32768, page=16, select=64, **QWEN),
        # 32 users, ragged contexts up to 32768, pages of 64
        dict(name="sparse_batch", op="sparse", seqs=32, context=32768, page=64, select=32, **QWEN),
        # 32 users of a 131072-token window, 2048 tokens attended each
        dict(name="sparse_window", op="sparse", seqs=32, context=131072, page=16, select=128, **QWEN),
        # 64-wide heads, a page size that is no power of two
        dict(name="sparse_d64", op="sparse", seqs=48, context=16000, page=48, select=21, **TINY),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append_mla", "shared", "shared", "summary", "sparse", "sparse"])
    heads = dict(rng.choice([QWEN, MHA, TINY, dict(H=8, G=4, d=128, base=5e5), dict(H=1, G=8, d=64, base=1e4)]))
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 10368), page=page, q=rng.random() < 0.7, **heads)
    if op == "append_mla":
        return dict(op=op, tokens=_log(rng, 1, 16381), page=page, lora=512, rope=64, Hq=rng.choice([0, 16, 128]),
                    base=1e4)
    if op == "summary":
        return dict(op=op, pages=_log(rng, 1, 8192), page=rng.choice([16, 32, 64]), **{**heads, "H": min(heads["H"], 8)})
    if op == "shared":
        seqs = _log(rng, 1, 64)
        top = min(98304, 64 * 98304 * 28 // (seqs * heads["H"] * heads["G"]))
        return dict(op=op, seqs=seqs, groups=rng.randint(1, min(seqs, 5)), prefix=_log(rng, 1, min(top, 32768)),
                    tail=_log(rng, 1, 1024), page=page, **heads)
    heads["H"] = min(heads["H"], 8)
    context = _log(rng, 1, 32768)
    pages = -(-context // page)
    return dict(op=op, seqs=_log(rng, 1, 32), context=context, page=page,
                select=rng.randint(2, max(2, min(128, pages))), **heads)


def _spread(n, most):
    """n ragged lengths up to ``most``: the first is the longest, one (of more than two) is empty."""
    out = [max(1, most - (most * ((5 * i) % n)) // (2 * n)) for i in range(n)]
    if n > 2:
        out[n // 2] = 0
    return out


def _group_start(seqs, groups):
    return [i * seqs // groups for i in range(groups + 1)]


def _prefixes(c):
    return [max(1, c["prefix"] - (c["prefix"] * i) // (4 * c["groups"])) for i in range(c["groups"])]


def _contexts(c):
    n = c["seqs"]
    return [max(1, c["context"] - (c["context"] * ((5 * i) % n)) // (4 * n)) for i in range(n)]


def work(c):
    if c["op"] == "append":
        row = (2 * c["H"] + (c["H"] * c["G"] if c["q"] else 0)) * c["d"] * 2
        turned = c["H"] + (c["H"] * c["G"] if c["q"] else 0)
        return {"bytes": c["tokens"] * (2 * row + 16), "flops": c["tokens"] * turned * c["d"] * 3}
    if c["op"] == "append_mla":
        row = (c["lora"] + c["rope"] + c["Hq"] * c["rope"]) * 2
        return {"bytes": c["tokens"] * (2 * row + 16), "flops": c["tokens"] * (1 + c["Hq"]) * c["rope"] * 3}
    if c["op"] == "summary":
        row = c["H"] * c["d"] * 2
        return {"bytes": c["pages"] * (c["page"] + 2) * row, "flops": c["pages"] * c["page"] * c["H"] * c["d"] * 2}
    H, G, d, n = c["H"], c["G"], c["d"], c["seqs"]
    io = n * H * G * (2 * d * 2 + 4)
    if c["op"] == "shared":
        starts, pre, tails = _group_start(n, c["groups"]), _prefixes(c), _spread(n, c["tail"])
        tokens = sum(pre) + sum(tails)
        seen = sum(tails) + sum((starts[g + 1] - starts[g]) * pre[g] for g in range(c["groups"]))
        return {"bytes": io + tokens * H * d * 4, "flops": 4 * d * H * G * seen}
    pages = [-(-x // c["page"]) for x in _contexts(c)]
    kept = sum(min(p, c["select"]) for p in pages)
    return {"bytes": io + sum(pages) * H * d * 4 + kept * H * c["page"] * d * 4 + 4 * n * H * c["select"],
            "flops": 4 * sum(pages) * H * d + 4 * d * H * G * kept * c["page"]}


# ----------------------------------------------------------------- inputs --
def _theta(base, rot):
    return base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64, device=DEV) / rot)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(1_000_003 * int(seed) + 17)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * std).to(torch.bfloat16)

    def permuted(n):
        return torch.randperm(n, generator=g, device=DEV).to(torch.int32)

    s = dict(c)
    if c["op"] in ("append", "append_mla"):
        T, P = c["tokens"], c["page"]
        n_pages = -(-T // P) + 4
        table = permuted(n_pages).long()
        t = torch.arange(T, device=DEV)
        s["slots"] = table[t // P] * P + t % P          # tokens fill pages in order, pages anywhere
        if T > 3:
            s["slots"][T // 2] = -1                     # a padded row of the batch
        start = torch.randint(0, 1 << 20, (1,), generator=g, device=DEV)
        s["positions"] = start + t
        if c["op"] == "append":
            H, G, d = c["H"], c["G"], c["d"]
            rows = normal(T, (H * G + 2 * H) * d)       # the fused projection's output: q | k | v
            s["rows_q"] = rows[:, :H * G * d].unflatten(1, (H * G, d)) if c["q"] else None
            s["rows_k"] = rows[:, H * G * d:(H * G + H) * d].unflatten(1, (H, d))
            s["rows_v"] = rows[:, (H * G + H) * d:].unflatten(1, (H, d))
            s["pool_k"], s["pool_v"] = normal(1, n_pages * P, H, d), normal(1, n_pages * P, H, d)
            s["q_out"] = torch.zeros(T, H * G, d, dtype=torch.bfloat16, device=DEV) if c["q"] else None
        else:
            r, W = c["rope"], c["lora"] + c["rope"]
            rows = normal(T, W)
            s["rows_c"], s["rows_r"] = rows[:, :c["lora"]], rows[:, c["lora"]:]
            s["rows_q"] = normal(T, c["Hq"], 128 + r)[:, :, 128:] if c["Hq"] else None
            s["pool"] = normal(1, n_pages * P, W)
            # the rope columns of the absorbed queries that attention reads
            s["q_out"] = torch.zeros(T, c["Hq"], W, dtype=torch.bfloat16, device=DEV) if c["Hq"] else None
        return s
    H, G, d, P = c["H"], c["G"], c["d"], c["page"]
    if c["op"] == "summary":
        n = c["pages"] + 4
        s["pool_k"] = normal(n * P, H, d)
        s["page_ids"] = permuted(n)[:c["pages"]].contiguous()
        s["page_tokens"] = torch.full((c["pages"],), P, dtype=torch.int32, device=DEV)
        s["page_tokens"][-1] = (P + 1) // 2             # the page still being filled
        s["summary"] = torch.zeros(n, H, 2, d, dtype=torch.bfloat16, device=DEV)
        return s
    n = c["seqs"]
    i32 = dict(dtype=torch.int32, device=DEV)

    def tables(lens, first):
        """Page tables of ``lens`` tokens each, drawn from the pool's pages from ``first`` on."""
        count = [-(-x // P) for x in lens]
        width = max(max(count), 1)
        at = torch.tensor([first + sum(count[:i]) for i in range(len(lens))], device=DEV)[:, None]
        k = torch.arange(width, device=DEV)[None]
        last = torch.tensor([max(x - 1, 0) for x in count], device=DEV)[:, None]
        return at + torch.minimum(k, last), first + sum(count)

    s["q"] = normal(n, H * G, d)
    if c["op"] == "shared":
        pre, tails = _prefixes(c), _spread(n, c["tail"])
        a, used = tables(pre, 0)
        b, used = tables(tails, used)
        order = permuted(used + 4)
        s["prefix_pages"], s["pages"] = order[a].contiguous(), order[torch.clamp(b, max=used + 3)].contiguous()
        s["prefix_len"], s["lens"] = torch.tensor(pre, **i32), torch.tensor(tails, **i32)
        starts = _group_start(n, c["groups"])
        s["group_start"] = torch.tensor(starts, **i32)
        s["max_group"] = max(starts[i + 1] - starts[i] for i in range(c["groups"]))
        s["max_prefix"], s["max_len"] = max(pre), max(tails)
        s["pool_k"], s["pool_v"] = normal((used + 4) * P, H, d), normal((used + 4) * P, H, d)
        return s
    lens = _contexts(c)
    a, used = tables(lens, 0)
    s["pages"] = permuted(used + 4)[a].contiguous()
    s["lens"], s["max_len"] = torch.tensor(lens, **i32), max(lens)
    # the keys of a page lie around a centre of its own, as those of neighbouring tokens do
    centre = torch.randn(used + 4, 1, H, d, generator=g, device=DEV) * 0.5
    s["pool_k"] = (torch.randn(used + 4, P, H, d, generator=g, device=DEV) * 0.7 + centre).to(torch.bfloat16)
    s["summary"] = torch.stack([s["pool_k"].amin(1), s["pool_k"].amax(1)], dim=2).contiguous()
    s["pool_k"] = s["pool_k"].view(-1, H, d)
    s["pool_v"] = normal((used + 4) * P, H, d)
    return s


# ------------------------------------------------------------- plain form --
def _turned(x, positions, base, interleaved):
    """x [T, heads, rot] turned by its positions; angles in 64 bits, the rotation in 32, one rounding."""
    ang = positions.double()[:, None] * _theta(base, x.shape[-1])
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    x = x.float()
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2).to(torch.bfloat16)
    a, b = x.chunk(2, dim=-1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1).to(torch.bfloat16)


def _put(rows, slots, values):
    """rows[slots] = values, leaving out slot -1 (its write goes to a row that stays as it is)."""
    keep = slots >= 0
    rows[slots[keep]] = values[keep]


def _rows_of(pages, page, count):
    """Slots of tokens 0 .. count-1 of each page table row."""
    t = torch.arange(count, device=DEV)
    return pages.long()[:, t // page] * page + t % page


def _softmax_parts(scores, seen):
    """Weights (unnormalised), row maximum and sum over the last axis where ``seen``; empty rows give zeros."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    safe = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    w = torch.exp(scores - safe)
    return w, safe[..., 0], w.sum(-1)


def _finish(o, top, total):
    some = total > 0
    out = torch.where(some[..., None], o / torch.where(some, total, torch.ones_like(total))[..., None],
                      torch.zeros_like(o))
    lse = torch.where(some, top + torch.log(torch.where(some, total, torch.ones_like(total))),
                      torch.full_like(total, -math.inf))
    return out, lse


def _plain_shared(s):
    n, H, G, d, P = s["seqs"], s["H"], s["G"], s["d"], s["page"]
    starts, M = s["group_start"].long(), s["max_group"]
    q = s["q"].float().view(n, H, G, d) * d ** -0.5
    # the sequences of a group side by side (padded), against the group's prefix once
    member = starts[:-1, None] + torch.arange(M, device=DEV)[None]
    real = member < starts[1:, None]
    qg = q[member.clamp(max=n - 1)]                                        # [groups, M, H, G, d]
    slots = _rows_of(s["prefix_pages"], P, s["max_prefix"])
    kp, vp = s["pool_k"][slots].float(), s["pool_v"][slots].float()        # [groups, prefix, H, d]
    seen = torch.arange(s["max_prefix"], device=DEV)[None] < s["prefix_len"][:, None]
    w, top, total = _softmax_parts(torch.einsum("bmhgd,bthd->bmhgt", qg, kp), seen[:, None, None, None])
    o = torch.einsum("bmhgt,bthd->bmhgd", w, vp)
    o1, top1, total1 = o[real], top[real], total[real]                     # [n, H, G, ...]: groups are in order
    slots = _rows_of(s["pages"], P, s["max_len"])
    kt, vt = s["pool_k"][slots].float(), s["pool_v"][slots].float()
    seen = torch.arange(s["max_len"], device=DEV)[None] < s["lens"][:, None]
    w, top2, total2 = _softmax_parts(torch.einsum("shgd,sthd->shgt", q, kt), seen[:, None, None])
    o2 = torch.einsum("shgt,sthd->shgd", w, vt)
    top1 = torch.where(total1 > 0, top1, torch.full_like(top1, -math.inf))
    top2 = torch.where(total2 > 0, top2, torch.full_like(top2, -math.inf))
    top = torch.maximum(top1, top2)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    f1, f2 = torch.exp(top1 - top), torch.exp(top2 - top)
    out, lse = _finish(o1 * f1[..., None] + o2 * f2[..., None], top, total1 * f1 + total2 * f2)
    return {"out": out.view(n, H * G, d).to(torch.bfloat16), "lse": lse.view(n, H * G)}


def _plain_select(s):
    n, H, G, d, P = s["seqs"], s["H"], s["G"], s["d"], s["page"]
    q = s["q"].double().view(n, H, G, d)
    count = (s["lens"].long() + P - 1) // P
    width = (s["max_len"] + P - 1) // P
    box = s["summary"][s["pages"][:, :width].long()]                       # [n, width, H, 2, d]
    # max(q mn, q mx) is q mx for q > 0 and q mn for q < 0, so the heads of a group add up first;
    # in 64 bits: the choice hangs on scores next to one another
    score = torch.einsum("shd,sjhd->shj", q.clamp(max=0).sum(2), box[:, :, :, 0].double()) \
        + torch.einsum("shd,sjhd->shj", q.clamp(min=0).sum(2), box[:, :, :, 1].double())
    j = torch.arange(width, device=DEV)[None]
    always = (j < 1) | (j >= count[:, None] - 1)
    score = torch.where(always[:, None], torch.full_like(score, math.inf), score)
    score = score.masked_fill((j >= count[:, None])[:, None], -math.inf)
    k = s["select"]
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :k]
    order = torch.nn.functional.pad(order, (0, k - order.shape[-1]), value=width)
    real = torch.arange(k, device=DEV) < torch.clamp(count, max=k)[:, None, None]
    order = torch.where(real, order, torch.full_like(order, 1 << 30)).sort(-1).values
    return torch.where(order < 1 << 30, order, torch.full_like(order, -1)).to(torch.int32)


def _plain_sparse(s):
    n, H, G, d, P = s["seqs"], s["H"], s["G"], s["d"], s["page"]
    chosen = _plain_select(s)
    j = chosen.long().clamp(min=0)                                         # [n, H, k]
    page = torch.gather(s["pages"].long()[:, None].expand(n, H, -1), 2, j)
    t = torch.arange(P, device=DEV)
    slots = (page[..., None] * P + t).flatten(2)                           # [n, H, k P]
    seen = ((chosen[..., None] >= 0) & (j[..., None] * P + t < s["lens"].long()[:, None, None, None])).flatten(2)
    head = torch.arange(H, device=DEV)[None, :, None]
    k, v = s["pool_k"][slots, head].float(), s["pool_v"][slots, head].float()
    q = s["q"].float().view(n, H, G, d) * d ** -0.5
    w, top, total = _softmax_parts(torch.einsum("shgd,shtd->shgt", q, k), seen[:, :, None])
    out, lse = _finish(torch.einsum("shgt,shtd->shgd", w, v), top, total)
    return {"out": out.view(n, H * G, d).to(torch.bfloat16), "lse": lse.view(n, H * G), "selected": chosen}


def _plain(s):
    if s["op"] == "append":
        _put(s["pool_k"][0], s["slots"], _turned(s["rows_k"], s["positions"], s["base"], False))
        _put(s["pool_v"][0], s["slots"], s["rows_v"])
        if s["q"]:
            keep = s["slots"] >= 0
            s["q_out"][keep] = _turned(s["rows_q"], s["positions"], s["base"], False)[keep]
        return {"pool_k": s["pool_k"], "pool_v": s["pool_v"], "q": s["q_out"]}
    if s["op"] == "append_mla":
        kr = _turned(s["rows_r"][:, None], s["positions"], s["base"], True)[:, 0]
        _put(s["pool"][0], s["slots"], torch.cat([s["rows_c"], kr], dim=1))
        if s["Hq"]:
            keep = s["slots"] >= 0
            s["q_out"][:, :, s["lora"]:][keep] = _turned(s["rows_q"], s["positions"], s["base"], True)[keep]
        return {"pool": s["pool"], "q": s["q_out"]}
    if s["op"] == "summary":
        P = s["page"]
        t = torch.arange(P, device=DEV)
        rows = s["pool_k"].view(-1, P, s["H"], s["d"])[s["page_ids"].long()].float()
        seen = (t[None] < s["page_tokens"][:, None])[:, :, None, None]
        low = rows.masked_fill(~seen, math.inf).amin(1)
        high = rows.masked_fill(~seen, -math.inf).amax(1)
        s["summary"][s["page_ids"].long()] = torch.stack([low, high], dim=2).to(torch.bfloat16)
        return {"summary": s["summary"]}
    return _plain_shared(s) if s["op"] == "shared" else _plain_sparse(s)


# -------------------------------------------------------------------- run --
def _own(s):
    import position_invariant_kv_chunk_gb300 as K

    if s["op"] == "append":
        K.kamera_append_kv(s["pool_k"], s["pool_v"], s["rows_k"], s["rows_v"], K.Rope(s["base"], s["d"]),
                           s["positions"], s["slots"], q=s["rows_q"], q_out=s["q_out"])
        return {"pool_k": s["pool_k"], "pool_v": s["pool_v"], "q": s["q_out"]}
    if s["op"] == "append_mla":
        out = None if s["q_out"] is None else s["q_out"][:, :, s["lora"]:]
        K.kamera_mla_append_kv(s["pool"], s["lora"], s["rows_c"], s["rows_r"],
                               K.Rope(s["base"], s["rope"], 0, K.INTERLEAVED), s["positions"], s["slots"],
                               q=s["rows_q"], q_out=out)
        return {"pool": s["pool"], "q": s["q_out"]}
    if s["op"] == "summary":
        K.kamera_summarize_pages(s["pool_k"], s["page"], s["page_ids"], s["page_tokens"], s["summary"])
        return {"summary": s["summary"]}
    if s["op"] == "shared":
        out, lse = K.kamera_attend_shared(s["pool_k"], s["pool_v"], s["q"], s["page"], s["group_start"],
                                          s["prefix_pages"], s["prefix_len"], s["pages"], s["lens"], s["max_group"],
                                          s["max_prefix"], s["max_len"])
        return {"out": out, "lse": lse}
    chosen = K.kamera_select_pages(s["q"], s["summary"], s["page"], s["pages"], s["lens"], s["max_len"], s["select"],
                                   n_first=1, n_last=1)
    out, lse = K.kamera_attend_selected(s["pool_k"], s["pool_v"], s["q"], s["page"], s["pages"], s["lens"], chosen,
                                        s["max_len"])
    return {"out": out, "lse": lse, "selected": chosen}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ exact --
def _exact_turn(x, p, base, pair):
    """Each pair of components as a complex number times e^(i p theta)."""
    r = x.shape[-1]
    x = x.to(torch.float64)
    lo = torch.arange(r // 2, device=DEV) * (2 if pair else 1)
    hi = lo + (1 if pair else r // 2)
    z = torch.complex(x[..., lo], x[..., hi])
    phase = p.to(torch.float64)[:, None, None] * torch.pow(
        torch.tensor(base, dtype=torch.float64, device=DEV), -torch.arange(0, r, 2, device=DEV).double() / r)
    z = z * torch.polar(torch.ones_like(phase), phase)
    y = torch.empty_like(x)
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _exact_attention(q, k, v):
    """One sequence and KV head: q [G, d], k and v [t, d] -> out [G, d], log-sum-exp [G]."""
    if k.shape[0] == 0:
        return torch.zeros_like(q), torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=DEV)
    z = (q @ k.t()) / math.sqrt(q.shape[1])
    return torch.softmax(z, dim=-1) @ v, torch.logsumexp(z, dim=-1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] in ("append", "append_mla"):
        kept = [i for i, x in enumerate(s["slots"].tolist()) if x >= 0]
        at, p = s["slots"][kept], s["positions"][kept]
        if c["op"] == "append":
            pk, pv = s["pool_k"].double(), s["pool_v"].double()
            pk[0, at] = _exact_turn(s["rows_k"][kept], p, c["base"], False)
            pv[0, at] = s["rows_v"][kept].double()
            q = None
            if c["q"]:
                q = s["q_out"].double()
                q[kept] = _exact_turn(s["rows_q"][kept], p, c["base"], False)
            return {"pool_k": pk, "pool_v": pv, "q": q}
        pool, q, lora = s["pool"].double(), None, c["lora"]
        pool[0, at, :lora] = s["rows_c"][kept].double()
        pool[0, at, lora:] = _exact_turn(s["rows_r"][kept][:, None], p, c["base"], True)[:, 0]
        if c["Hq"]:
            q = s["q_out"].double()
            q[kept, :, lora:] = _exact_turn(s["rows_q"][kept], p, c["base"], True)
        return {"pool": pool, "q": q}
    H, G, d, P = c["H"], c["G"], c["d"], c["page"]
    if c["op"] == "summary":
        out = s["summary"].double()
        ids, tokens = s["page_ids"].tolist(), s["page_tokens"].tolist()
        for page, count in zip(ids, tokens):
            rows = s["pool_k"][page * P:page * P + count].double()
            out[page, :, 0], out[page, :, 1] = rows.min(0).values, rows.max(0).values
        return {"summary": out}
    n = c["seqs"]
    out = torch.empty(n, H * G, d, dtype=torch.float64, device=DEV)
    lse = torch.empty(n, H * G, dtype=torch.float64, device=DEV)
    lens = s["lens"].tolist()

    def slots(table, count):
        t = torch.arange(count, device=DEV)
        return table.long()[t // P] * P + t % P

    if c["op"] == "shared":
        starts, pre = s["group_start"].tolist(), s["prefix_len"].tolist()
        for g in range(c["groups"]):
            a = slots(s["prefix_pages"][g], pre[g])
            for h in range(H):
                kp, vp = s["pool_k"][a, h].double(), s["pool_v"][a, h].double()
                for i in range(starts[g], starts[g + 1]):
                    b = slots(s["pages"][i], lens[i])
                    r = slice(h * G, h * G + G)
                    out[i, r], lse[i, r] = _exact_attention(
                        s["q"][i, r].double(), torch.cat([kp, s["pool_k"][b, h].double()]),
                        torch.cat([vp, s["pool_v"][b, h].double()]))
        return {"out": out, "lse": lse}
    chosen = torch.full((n, H, c["select"]), -1, dtype=torch.int64, device=DEV)
    for i in range(n):
        count = -(-lens[i] // P)
        box = s["summary"][s["pages"][i, :count].long()].double()          # [count, H, 2, d]
        for h in range(H):
            q = s["q"][i, h * G:h * G + G].double()
            best = torch.maximum(q[:, None] * box[None, :, h, 0], q[:, None] * box[None, :, h, 1]).sum((0, 2))
            best[0] = best[count - 1] = math.inf
            rank = sorted(range(count), key=lambda j, b=best.tolist(): (-b[j], j))[:c["select"]]
            rank = torch.tensor(sorted(rank), device=DEV)
            chosen[i, h, :len(rank)] = rank
            t = (rank[:, None] * P + torch.arange(P, device=DEV)).flatten()
            t = t[t < lens[i]]
            a = s["pages"][i].long()[t // P] * P + t % P
            r = slice(h * G, h * G + G)
            out[i, r], lse[i, r] = _exact_attention(q, s["pool_k"][a, h].double(), s["pool_v"][a, h].double())
    return {"out": out, "lse": lse, "selected": chosen}
