"""Measured cases of latent attention over the paged MLA pool (absorbed decode, expansion of latent rows,
attention over expanded rows) and of the 4-bit pool (packing cold pages, attention that reads them).

Each case names its operator in ``op``; ``prepare`` draws what a serving loop holds before the call,
``run`` makes one pass (the plain form in elementary torch operations, or the library's entry points
when ``own`` is set), ``exact`` states the same result from the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
LORA, ROPE, NOPE, VDIM = 512, 64, 128, 128   # DeepSeek-V2 shaped latent rows and heads
QWEN = dict(H=4, G=7, d=128)                 # Qwen2.5-VL-7B shaped heads: 28 query heads on 4 KV heads
MHA = dict(H=32, G=1, d=128)                 # the MHA workload's 32 heads
TINY = dict(H=2, G=4, d=64)                  # 2 KV heads of 64


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one user's decode step over a 4096-token latent cache (latency)
        dict(name="mla_one", op="mla_decode", seqs=1, context=4096, page=16, Hq=16),
        # 32 users, ragged contexts up to 16384, 16 heads on one latent row
        dict(name="mla_batch", op="mla_decode", seqs=32, context=16384, page=64, Hq=16),
        # 48 users of a model with 128 heads: as many flops as bytes allow
        dict(name="mla_wide", op="mla_decode", seqs=48, context=8192, page=64, Hq=128),
        # a recalled 1296-token frame, its latent rows expanded before a prefill reads them
        dict(name="expand_frame", op="mla_expand", tokens=1296, page=16, Hq=16),
        # a long prompt's rows expanded at once
        dict(name="expand_prompt", op="mla_expand", tokens=16381, page=64, Hq=16),
        # a question of 777 tokens behind a recalled frame
        dict(name="prefill_question", op="mla_prefill", seqs=1, new=777, prefix=1296, Hq=16),
        # four prompts of up to 4096 tokens, nothing before them
        dict(name="prefill_prompts", op="mla_prefill", seqs=4, new=4096, prefix=0, Hq=16),
        # the pages that 64 sequences have just filled, to 4 bits and back (latency)
        dict(name="pack_step", op="pack", pages=64, page=16, **QWEN),
        # 65536 cold tokens at once
        dict(name="pack_cold", op="pack", pages=4096, page=16, **QWEN),
        # one user, 32768 tokens in 4 bits and the page being filled in bf16 (latency)
        dict(name="packed_one", op="packed", seqs=1, context=32768, tail=13, page=16, **QWEN),
        # 32 users of up to 32768 tokens
        dict(name="packed_batch", op="packed", seqs=32, context=32768, tail=64, page=64, **QWEN),
        # MHA heads, every head with keys of its own
        dict(name="packed_mha", op="packed", seqs=8, context=8192, tail=37, page=64, **MHA),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["mla_decode", "mla_decode", "mla_expand", "mla_prefill", "mla_prefill", "pack", "packed", "packed"])
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "mla_decode":
        return dict(op=op, seqs=_log(rng, 1, 48), context=_log(rng, 1, 8192), page=page,
                    Hq=rng.choice([1, 8, 16, 20, 32, 40, 64, 128]))
    if op == "mla_expand":
        return dict(op=op, tokens=_log(rng, 1, 16381), page=page, Hq=rng.choice([4, 8, 16]))
    if op == "mla_prefill":
        return dict(op=op, seqs=rng.randint(1, 4), new=_log(rng, 1, 2900), prefix=rng.choice([0, _log(rng, 1, 2900)]),
                    Hq=rng.choice([4, 8, 16]))
    heads = dict(rng.choice([QWEN, MHA, TINY, dict(H=8, G=4, d=128), dict(H=2, G=12, d=128), dict(H=1, G=8, d=64)]))
    if op == "pack":
        return dict(op=op, pages=_log(rng, 1, 4096 * 16 * 4 // (page * heads["H"])), page=page, **heads)
    seqs = _log(rng, 1, 32)
    top = 32 * 32768 * 4 // (seqs * heads["H"])
    return dict(op=op, seqs=seqs, context=_log(rng, 1, min(32768, top)), tail=rng.choice([0, rng.randint(1, 2 * page)]),
                page=page, **heads)


def _ragged(n, most):
    """n ragged lengths up to ``most``: the first is the longest, one (of more than two) is empty."""
    out = [max(1, most - (most * ((5 * i) % n)) // (4 * n)) for i in range(n)]
    if n > 2:
        out[n // 2] = 0
    return out


def _tails(c):
    n = c["seqs"]
    return [c["tail"] * (n - i) // n for i in range(n)]


def _new(c):
    n = c["seqs"]
    return [max(1, c["new"] - (c["new"] * i) // (3 * n)) for i in range(n)]


def _prefix(c):
    n = c["seqs"]
    return [c["prefix"] - (c["prefix"] * ((3 * i) % n)) // (2 * n) for i in range(n)]


def work(c):
    if c["op"] == "mla_decode":
        t, rows, W = sum(_ragged(c["seqs"], c["context"])), c["seqs"] * c["Hq"], LORA + ROPE
        return {"bytes": 2 * W * t + rows * (2 * W + 2 * LORA + 4) + 4 * (t // c["page"] + 2 * c["seqs"]),
                "flops": 2 * c["Hq"] * (W + LORA) * t}
    if c["op"] == "mla_expand":
        T, N = c["tokens"], c["Hq"] * (NOPE + VDIM)
        return {"bytes": T * (2 * (LORA + 2 * ROPE) + 8 + 2 * N) + 2 * N * LORA, "flops": 2 * T * N * LORA}
    if c["op"] == "mla_prefill":
        q, k = _new(c), [a + b for a, b in zip(_prefix(c), _new(c))]
        pairs = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(q, k))
        return {"bytes": c["Hq"] * (sum(q) * (2 * (NOPE + ROPE + VDIM) + 4) + sum(k) * 2 * (NOPE + VDIM))
                + sum(k) * 2 * ROPE, "flops": 2 * c["Hq"] * (NOPE + ROPE + VDIM) * pairs}
    H, G, d = c["H"], c["G"], c["d"]
    if c["op"] == "pack":
        t = c["pages"] * c["page"] * H
        return {"bytes": t * (2 * 4 * d + 2 * (d + d // 8)) + 12 * c["pages"], "flops": 8 * t * d}
    t, tail, rows = sum(_ragged(c["seqs"], c["context"])), sum(_tails(c)), c["seqs"] * H * G
    return {"bytes": H * (t * (d + d // 8) + tail * 4 * d) + rows * (4 * d + 4) + 4 * ((t + tail) // c["page"]),
            "flops": 4 * H * G * d * (t + tail)}


# ------------------------------------------------------------------ inputs --
def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    i32 = dict(dtype=torch.int32, device=DEV)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * std).to(torch.bfloat16)

    def permuted(n):
        return torch.randperm(n, generator=g, device=DEV).to(torch.int32)

    def tables(lens, P):
        """Page tables of ``lens`` tokens each over pages in any order, and how many pages there are."""
        count = [-(-x // P) for x in lens]
        at = torch.tensor([sum(count[:i]) for i in range(len(lens))], device=DEV)[:, None]
        k = torch.arange(max(max(count), 1), device=DEV)[None]
        last = torch.tensor([max(x - 1, 0) for x in count], device=DEV)[:, None]
        n = sum(count) + 4
        return permuted(n)[torch.clamp(at + torch.minimum(k, last), max=n - 1)].contiguous(), n

    s = dict(c)
    if c["op"] == "mla_decode":
        lens = _ragged(c["seqs"], c["context"])
        s["pages"], n = tables(lens, c["page"])
        s["lens"], s["max_len"] = torch.tensor(lens, **i32), max(lens)
        s["pool"] = normal(n * c["page"], LORA + ROPE)
        s["q"] = normal(c["seqs"], c["Hq"], LORA + ROPE)
        return s
    if c["op"] == "mla_expand":
        T, P = c["tokens"], c["page"]
        n = -(-T // P) + 4
        t = torch.arange(T, device=DEV)
        s["slots"] = permuted(n).long()[t // P] * P + t % P
        s["pool"] = normal(n * P, LORA + ROPE)
        s["weight"] = normal(c["Hq"], NOPE + VDIM, LORA, std=LORA ** -0.5)
        return s
    if c["op"] == "mla_prefill":
        q, k = _new(c), [a + b for a, b in zip(_prefix(c), _new(c))]
        s["q"] = normal(sum(q), c["Hq"], NOPE + ROPE)
        s["kv"] = normal(sum(k), c["Hq"], NOPE + VDIM)
        s["k_rope"] = normal(sum(k), ROPE)
        s["q_start"] = torch.tensor([sum(q[:i]) for i in range(len(q) + 1)], **i32)
        s["kv_start"] = torch.tensor([sum(k[:i]) for i in range(len(k) + 1)], **i32)
        s["max_q"], s["max_kv"] = max(q), max(k)
        return s
    H, G, d, P = c["H"], c["G"], c["d"], c["page"]
    if c["op"] == "pack":
        n = c["pages"] + 4
        s["src"], s["dst"] = permuted(n)[:c["pages"]].contiguous(), permuted(n)[:c["pages"]].contiguous()
        s["tokens"] = torch.full((c["pages"],), P, **i32)
        s["tokens"][-1] = (P + 1) // 2                  # a page that its sequence ended in
        s["pool_k"], s["pool_v"] = normal(n * P, H, d), normal(n * P, H, d, std=0.5)
        s["back_k"], s["back_v"] = torch.zeros_like(s["pool_k"]), torch.zeros_like(s["pool_v"])
        s["packed"] = torch.zeros(n, H, P * (d + d // 8), dtype=torch.uint8, device=DEV)
        return s
    lens, tails = _ragged(c["seqs"], c["context"]), _tails(c)
    s["pages"], n = tables(lens, P)
    s["lens"], s["max_len"] = torch.tensor(lens, **i32), max(lens)
    s["q"] = normal(c["seqs"], H * G, d)
    whole, every = torch.full((n,), P, **i32), torch.arange(n, **i32)
    pool_k, pool_v = normal(n * P, H, d), normal(n * P, H, d)
    if own:
        import position_invariant_kv_chunk_gb300 as K
        s["packed"] = torch.zeros(n, H, P * (d + d // 8), dtype=torch.uint8, device=DEV)
        K.kamera_pack_pages(pool_k, pool_v, P, every, whole, s["packed"], every)
    # the same cache as codes (two to a byte) and scales, which the plain form reads
    s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"] = [], [], [], []
    for i in range(0, n, 2048):
        k = pool_k[i * P:(i + 2048) * P].view(-1, P, H, d)
        v = pool_v[i * P:(i + 2048) * P].view(-1, P, H, d)
        for x, name in ((_key_groups(k), "k"), (_value_groups(v), "v")):
            scale, code = _quantised(x)
            s[name + "_codes"].append((code[..., 0::2] | code[..., 1::2] << 4).to(torch.uint8))
            s[name + "_scales"].append(scale.to(torch.float8_e4m3fn))
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        s[name] = torch.cat([x.view(torch.uint8) for x in s[name]])
    del pool_k, pool_v
    s["tail_pages"], m = tables(tails, P)
    s["tail_lens"], s["max_tail"] = torch.tensor(tails, **i32), max(tails)
    s["pool_k"], s["pool_v"] = normal(m * P, H, d), normal(m * P, H, d)
    return s


# ------------------------------------------------------ the 4-bit format --
# 16 values share a scale in 8 bits (e4m3); a value is one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 times it.
# Keys are grouped along their channels, values along 16 tokens of a page: the axis that is summed over.
def _key_groups(k):
    """[pages, P, H, d] -> [pages, P, H, d / 16, 16]"""
    return k.unflatten(3, (-1, 16))


def _value_groups(v):
    """[pages, P, H, d] -> [pages, P / 16, H, d, 16]"""
    return v.unflatten(1, (-1, 16)).permute(0, 1, 3, 4, 2)


def _quantised(x):
    """Groups of 16 (the last axis) to their scale (fp32, an e4m3 value) and codes 0-15 (bit 3: the sign)."""
    x = x.float()
    scale = (x.abs().amax(-1) / 6).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    a, t = x.abs(), scale[..., None]
    code = torch.zeros_like(x, dtype=torch.int32)
    # halfway goes to the even code: up from codes 1, 3, 5, down from 0, 2, 4, 6
    for border, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += ((a >= border * t) if up else (a > border * t)).int()
    code = torch.where(t > 0, code, torch.zeros_like(code))
    return scale, code + 8 * (x < 0).int()


def _values(code, scale):
    level = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
    return torch.where(code >= 8, -level[code & 7], level[code & 7]) * scale[..., None]


def _read(codes, scales):
    """Groups of 16 values (fp32) out of packed codes and scale bytes."""
    code = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).long()
    return _values(code, scales.view(torch.float8_e4m3fn).float())


# ------------------------------------------------------------- plain form --
def _slots(row, page, n):
    t = torch.arange(n, device=DEV)
    return row.long()[t // page] * page + t % page


def _softmax(scores):
    """Weights over the last axis and the log of their sum; a row of -inf gives zeros and -inf."""
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    w = torch.exp(scores - top)
    total = w.sum(-1, keepdim=True)
    some = total > 0
    one = torch.where(some, total, torch.ones_like(total))
    return w / one, torch.where(some, top + torch.log(one), torch.full_like(total, -math.inf))[..., 0]


def _plain_decode(s):
    out = torch.zeros(s["seqs"], s["Hq"], LORA, device=DEV)
    lse = torch.full((s["seqs"], s["Hq"]), -math.inf, device=DEV)
    # short contexts side by side would pad; each sequence reads its own rows once
    for i, n in enumerate(_ragged(s["seqs"], s["context"])):
        if n > 0:
            row = s["pool"][_slots(s["pages"][i], s["page"], n)].float()
            w, lse[i] = _softmax((s["q"][i].float() * (LORA + ROPE) ** -0.5) @ row.T)
            out[i] = w @ row[:, :LORA]
    return {"out": out.to(torch.bfloat16), "lse": lse}


def _plain_expand(s):
    row = s["pool"][s["slots"]]
    kv = row[:, :LORA].float() @ s["weight"].flatten(0, 1).float().T
    return {"kv": kv.to(torch.bfloat16).unflatten(1, (s["Hq"], -1)), "k_rope": row[:, LORA:].contiguous()}


def _plain_prefill(s):
    T, Hq = s["q"].shape[:2]
    out = torch.zeros(T, Hq, VDIM, dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros(T, Hq, device=DEV)
    q0 = k0 = 0
    for new, pre in zip(_new(s), _prefix(s)):
        nk = new + pre
        q = s["q"][q0:q0 + new].float().transpose(0, 1) * (NOPE + ROPE) ** -0.5          # [Hq, new, 192]
        kv = s["kv"][k0:k0 + nk].float().transpose(0, 1)                                  # [Hq, nk, 256]
        scores = q[..., :NOPE] @ kv[..., :NOPE].transpose(1, 2) + q[..., NOPE:] @ s["k_rope"][k0:k0 + nk].float().T
        hidden = torch.arange(nk, device=DEV)[None] > torch.arange(new, device=DEV)[:, None] + pre
        w, l = _softmax(scores.masked_fill(hidden, -math.inf))
        out[q0:q0 + new] = (w @ kv[..., NOPE:]).transpose(0, 1).to(torch.bfloat16)
        lse[q0:q0 + new] = l.T
        q0, k0 = q0 + new, k0 + nk
    return {"out": out, "lse": lse}


def _plain_pack(s):
    P, H, d = s["page"], s["H"], s["d"]
    src, dst = s["src"].long(), s["dst"].long()
    there = (torch.arange(P, device=DEV)[None] < s["tokens"][:, None])[..., None, None]
    zero = torch.zeros((), dtype=torch.bfloat16, device=DEV)
    k = torch.where(there, s["pool_k"].view(-1, P, H, d)[src], zero)
    v = torch.where(there, s["pool_v"].view(-1, P, H, d)[src], zero)
    scale, code = _quantised(_key_groups(k))
    k = _values(code.long(), scale).flatten(3).to(torch.bfloat16)
    scale, code = _quantised(_value_groups(v))
    v = _values(code.long(), scale).permute(0, 1, 4, 2, 3).flatten(1, 2).to(torch.bfloat16)
    bk, bv = s["back_k"].view(-1, P, H, d), s["back_v"].view(-1, P, H, d)
    bk[dst], bv[dst] = torch.where(there, k, bk[dst]), torch.where(there, v, bv[dst])
    return {"k": s["back_k"], "v": s["back_v"]}


def _plain_packed(s):
    n, H, G, d, P = s["seqs"], s["H"], s["G"], s["d"], s["page"]
    out = torch.zeros(n, H, G, d, device=DEV)
    lse = torch.full((n, H, G), -math.inf, device=DEV)
    for i, (a, b) in enumerate(zip(_ragged(n, s["context"]), _tails(s))):
        if a + b == 0:
            continue
        ids = s["pages"][i, :-(-a // P)].long()
        k = _read(s["k_codes"][ids], s["k_scales"][ids]).flatten(3).flatten(0, 1)[:a]
        v = _read(s["v_codes"][ids], s["v_scales"][ids]).permute(0, 1, 4, 2, 3).flatten(0, 2)[:a]
        t = _slots(s["tail_pages"][i], P, b)
        k = torch.cat([k, s["pool_k"][t].float()]).transpose(0, 1)                        # [H, a + b, d]
        v = torch.cat([v, s["pool_v"][t].float()]).transpose(0, 1)
        w, lse[i] = _softmax((s["q"][i].float().view(H, G, d) * d ** -0.5) @ k.transpose(1, 2))
        out[i] = w @ v
    return {"out": out.to(torch.bfloat16).flatten(1, 2), "lse": lse.flatten(1)}


def run(s):
    if not own:
        return {"mla_decode": _plain_decode, "mla_expand": _plain_expand, "mla_prefill": _plain_prefill,
                "pack": _plain_pack, "packed": _plain_packed}[s["op"]](s)
    import position_invariant_kv_chunk_gb300 as K
    if s["op"] == "mla_decode":
        out, lse = K.kamera_mla_attend_paged(s["pool"], LORA, s["q"], s["page"], s["pages"], s["lens"], s["max_len"])
        return {"out": out, "lse": lse}
    if s["op"] == "mla_expand":
        kv, k_rope = K.kamera_mla_expand(s["pool"], LORA, s["weight"], s["slots"])
        return {"kv": kv, "k_rope": k_rope}
    if s["op"] == "mla_prefill":
        out, lse = K.kamera_mla_prefill_attend(s["q"], s["kv"], s["k_rope"], s["q_start"], s["kv_start"], s["max_q"],
                                               s["max_kv"])
        return {"out": out, "lse": lse}
    if s["op"] == "pack":
        K.kamera_pack_pages(s["pool_k"], s["pool_v"], s["page"], s["src"], s["tokens"], s["packed"], s["dst"])
        K.kamera_unpack_pages(s["packed"], s["page"], s["dst"], s["tokens"], s["back_k"], s["back_v"], s["dst"])
        return {"k": s["back_k"], "v": s["back_v"]}
    out, lse = K.kamera_attend_packed(s["packed"], s["q"], s["page"], s["pages"], s["lens"], s["max_len"],
                                      s["pool_k"], s["pool_v"], s["tail_pages"], s["tail_lens"], s["max_tail"])
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ exact --
def _attended(scores, values):
    """Softmax of 64-bit scores [..., n] over values [..., n, d], with its log-sum-exp."""
    lse = torch.logsumexp(scores, -1)
    return torch.exp(scores - lse[..., None]) @ values, lse


def _nearest(x):
    """Groups of 16 bf16 numbers to what 4 bits and their scale hold, in 64 bits, from the format's definition:
    each number to the nearest of the group's 15 levels, an even code where two are as near."""
    x = x.double()
    want = x.abs().amax(-1) / 6
    # e4m3: 3 bits behind the leading one, steps of 2^-9 below 2^-6, 448 at the most
    step = torch.exp2(torch.floor(torch.log2(want.clamp(min=2.0 ** -6))) - 3)
    scale = (torch.round(want / step) * step).clamp(max=448.0)[..., None]
    level = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=DEV)
    far = (x.abs()[..., None] - level * scale[..., None]).abs()
    odd = torch.arange(8, device=DEV) % 2
    best = far.amin(-1, keepdim=True)
    code = torch.where(far == best, odd, torch.full_like(odd, 2)).argmin(-1)
    return torch.where(x < 0, -1.0, 1.0) * level[code] * scale


def exact(c, seed):
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    P = c.get("page")
    if c["op"] == "mla_decode":
        out = torch.zeros(c["seqs"], c["Hq"], LORA, dtype=torch.float64, device=DEV)
        lse = torch.full((c["seqs"], c["Hq"]), -math.inf, dtype=torch.float64, device=DEV)
        for i, n in enumerate(s["lens"].tolist()):
            if n > 0:
                t = torch.arange(n, device=DEV)
                row = s["pool"][s["pages"][i].long()[t // P] * P + t % P].double()
                out[i], lse[i] = _attended(s["q"][i].double() @ row.T / math.sqrt(LORA + ROPE), row[:, :LORA])
        return {"out": out, "lse": lse}
    if c["op"] == "mla_expand":
        row = s["pool"].index_select(0, s["slots"]).double()
        kv = torch.stack([row[:, :LORA] @ w.double().T for w in s["weight"]], dim=1)
        return {"kv": kv, "k_rope": row[:, LORA:]}
    if c["op"] == "mla_prefill":
        T, Hq = s["q"].shape[:2]
        out = torch.zeros(T, Hq, VDIM, dtype=torch.float64, device=DEV)
        lse = torch.zeros(T, Hq, dtype=torch.float64, device=DEV)
        qs, ks = s["q_start"].tolist(), s["kv_start"].tolist()
        for i in range(c["seqs"]):
            nq, nk = qs[i + 1] - qs[i], ks[i + 1] - ks[i]
            seen = torch.ones(nq, nk, dtype=torch.bool, device=DEV).tril(nk - nq)
            for h in range(Hq):
                k = torch.cat([s["kv"][ks[i]:ks[i + 1], h, :NOPE], s["k_rope"][ks[i]:ks[i + 1]]], dim=1).double()
                score = s["q"][qs[i]:qs[i + 1], h].double() @ k.T / math.sqrt(NOPE + ROPE)
                score[~seen] = -math.inf
                out[qs[i]:qs[i + 1], h], lse[qs[i]:qs[i + 1], h] = \
                    _attended(score, s["kv"][ks[i]:ks[i + 1], h, NOPE:].double())
        return {"out": out, "lse": lse}
    H, G, d = c["H"], c["G"], c["d"]
    if c["op"] == "pack":
        k, v = s["back_k"].double(), s["back_v"].double()
        src, dst, count = s["src"].long(), s["dst"].long(), s["tokens"].tolist()
        pk, pv = s["pool_k"].view(-1, P, H, d), s["pool_v"].view(-1, P, H, d)
        for i in range(0, len(count), 256):
            a, n = src[i:i + 256], torch.tensor(count[i:i + 256], device=DEV)
            gone = torch.arange(P, device=DEV)[None] >= n[:, None]
            x, y = pk[a].clone(), pv[a].clone()
            x[gone], y[gone] = 0, 0
            x = _nearest(x.reshape(-1, 16)).view(-1, P, H, d)
            y = _nearest(y.view(-1, P // 16, 16, H, d).movedim(2, -1).reshape(-1, 16))
            y = y.view(-1, P // 16, H, d, 16).movedim(-1, 2).reshape(-1, P, H, d)
            b = dst[i:i + 256]
            k.view(-1, P, H, d)[b] = torch.where(gone[..., None, None], k.view(-1, P, H, d)[b], x)
            v.view(-1, P, H, d)[b] = torch.where(gone[..., None, None], v.view(-1, P, H, d)[b], y)
        return {"k": k, "v": v}
    out = torch.zeros(c["seqs"], H * G, d, dtype=torch.float64, device=DEV)
    lse = torch.full((c["seqs"], H * G), -math.inf, dtype=torch.float64, device=DEV)
    level = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=DEV)
    level = torch.cat([level, -level])
    lens, tails = s["lens"].tolist(), s["tail_lens"].tolist()

    def numbers(name, ids, h):
        """The groups of 16 of one head of some pages."""
        byte = s[name + "_codes"][ids][:, :, h]
        scale = s[name + "_scales"][ids][:, :, h].view(torch.float8_e4m3fn).double()[..., None]
        return torch.stack([level[(byte % 16).long()], level[(byte // 16).long()]], dim=-1).flatten(-2) * scale

    for i in range(c["seqs"]):
        if lens[i] + tails[i] == 0:
            continue
        ids = s["pages"][i, :(lens[i] + P - 1) // P].long()
        t = torch.arange(tails[i], device=DEV)
        t = s["tail_pages"][i].long()[t // P] * P + t % P
        for h in range(H):
            k = numbers("k", ids, h).reshape(-1, d)[:lens[i]]
            v = numbers("v", ids, h).movedim(-1, 2).reshape(-1, d)[:lens[i]]
            k, v = torch.cat([k, s["pool_k"][t, h].double()]), torch.cat([v, s["pool_v"][t, h].double()])
            r = slice(h * G, h * G + G)
            out[i, r], lse[i, r] = _attended(s["q"][i, r].double() @ k.T / math.sqrt(d), v)
    return {"out": out, "lse": lse}
