"""kamera_append_kv and kamera_mla_append_kv against their definitions in 64 bits.

Tolerance of a rotated component: its rounding to bf16, half a step = 2^-8
relative, plus fp32 work on the pair (a, b): the angle in half-turns carries
one fp32 rounding (2^-24 relative of at most one half-turn, 2^-24 pi radians),
cos and sin about 2 ulp each (2^-22), two products and a sum (3 x 2^-24), in all
below 2^-20 (|a| + |b|).  Copies are exact."""
import numpy as np
import pytest
import torch

import position_invariant_kv_chunk_gb300 as K
import workloads as W
from tests import paged_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
SLOT, DESCRIPTOR = 1, 4


def near(got: torch.Tensor, ref: np.ndarray, pair: np.ndarray, what):
    """Rotated rows within the tolerance; components outside the rotary range equal."""
    g = R.f64(got)
    err = np.abs(g - ref)
    ok = err <= R.ulp_half(ref) + 2.0 ** -20 * pair * (1 + 2.0 ** -8)
    assert ok.all(), (what, float(err[~ok].max()))
    still = pair == 0
    assert np.array_equal(g[still], ref[still]), what


def normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=DEV).to(torch.bfloat16)


CASES = {
    # T, H, Hq, d, rot, off, interleaved
    "qwen_step": (3, 4, 28, 128, 128, 0, False),
    "one_token": (1, 2, 8, 64, 64, 0, False),
    "mha_prompt": (700, 32, 32, 128, 128, 0, False),
    "long_prompt": (2600, 2, 4, 64, 64, 0, False),
    "partial_half": (37, 3, 5, 80, 48, 8, False),
    "partial_interleaved": (37, 2, 2, 96, 40, 16, True),
    "interleaved": (650, 1, 1, 64, 64, 0, True),
    "no_rotation": (9, 2, 4, 64, 0, 0, False),
    "no_query": (11, 2, 0, 128, 128, 0, False),
    "wide": (5, 1, 3, 512, 256, 8, False),
}


@pytest.mark.parametrize("name", list(CASES))
def test_append_matches_definition(name):
    T, H, Hq, d, rot, off, il = CASES[name]
    g = torch.Generator(device=DEV).manual_seed(len(name) * 131 + T)
    L, S, layer = 3, T + 40, 1
    pk, pv = normal(g, L, S, H, d), normal(g, L, S, H, d)
    fused = normal(g, T, (Hq + 2 * H) * d + 8)          # views of one projection, an odd row stride
    q = fused[:, :Hq * d].unflatten(1, (Hq, d)) if Hq else None
    k = fused[:, Hq * d:(Hq + H) * d].unflatten(1, (H, d))
    v = fused[:, (Hq + H) * d:(Hq + 2 * H) * d].unflatten(1, (H, d))
    slots = torch.randperm(S, generator=g, device=DEV)[:T].contiguous()
    if T > 2:
        slots[T // 2] = -1
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device=DEV)
    pos[0] = 0
    pos[-1] = 2 ** 31 - 1
    if T > 4:
        pos[1] = -(2 ** 31 - 1)
    before_k, before_v = pk.clone(), pv.clone()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    q_out = torch.full((T, Hq, d), 7.0, dtype=torch.bfloat16, device=DEV) if Hq else None
    got = K.kamera_append_kv(pk, pv, k, v, K.Rope(1e4, rot, off, K.INTERLEAVED if il else K.ROTATE_HALF), pos, slots,
                             layer=layer, q=q, q_out=q_out, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert got is q_out
    kept = (slots >= 0).cpu().numpy()
    at = slots[slots >= 0]
    inv = 1e4 ** (-2.0 * np.arange(rot // 2) / rot) if rot else np.zeros(0)
    p = pos.cpu().numpy()[kept]
    xk = R.f64(k)[kept]
    near(pk[layer, at], R.turned(xk, p, inv, off, il), R.turn_scale(xk, rot // 2, off, il), name)
    assert torch.equal(pv[layer, at], v[slots >= 0])
    if Hq:
        xq = R.f64(q)[kept]
        near(q_out[torch.from_numpy(kept).to(DEV)], R.turned(xq, p, inv, off, il),
             R.turn_scale(xq, rot // 2, off, il), name)
        assert bool((q_out[slots < 0] == 7).all()), "a padding row's query was written"
    # every other slot and layer stays as it was
    before_k[layer, at], before_v[layer, at] = pk[layer, at], pv[layer, at]
    assert torch.equal(pk, before_k) and torch.equal(pv, before_v)


@pytest.mark.parametrize("T,Hq", [(5, 16), (1, 128), (1300, 0)])
def test_mla_append_matches_definition(T, Hq):
    g = torch.Generator(device=DEV).manual_seed(T + Hq)
    lora, rd, S = 512, 64, T + 9
    pool = normal(g, 2, S, lora + rd)
    rows = normal(g, T, lora + rd)
    full = normal(g, T, Hq, 128 + rd) if Hq else None
    out = torch.zeros(T, Hq, lora + rd, dtype=torch.bfloat16, device=DEV) if Hq else None
    slots = torch.randperm(S, generator=g, device=DEV)[:T].contiguous()
    pos = torch.randint(0, 200000, (T,), generator=g, device=DEV)
    before = pool.clone()
    K.kamera_mla_append_kv(pool, lora, rows[:, :lora], rows[:, lora:], K.Rope(1e4, rd, 0, K.INTERLEAVED), pos, slots,
                           layer=1, q=full[:, :, 128:] if Hq else None, q_out=out[:, :, lora:] if Hq else None)
    torch.cuda.synchronize()
    inv = 1e4 ** (-2.0 * np.arange(rd // 2) / rd)
    p = pos.cpu().numpy()
    assert torch.equal(pool[1, slots, :lora], rows[:, :lora])
    x = R.f64(rows[:, None, lora:])
    near(pool[1, slots][:, None, lora:], R.turned(x, p, inv, 0, True), R.turn_scale(x, rd // 2, 0, True), "k_rope")
    if Hq:
        x = R.f64(full[:, :, 128:])
        near(out[:, :, lora:], R.turned(x, p, inv, 0, True), R.turn_scale(x, rd // 2, 0, True), "q")
        assert not bool(out[:, :, :lora].any()), "the latent columns of the queries were written"
    before[1, slots] = pool[1, slots]
    assert torch.equal(pool, before)


@pytest.mark.parametrize("layout", ["sections", "interleaved"])
def test_append_multi_axis_positions(layout):
    T, H, d = 21, 2, 128
    g = torch.Generator(device=DEV).manual_seed(3)
    pk, pv = normal(g, 1, 64, H, d), normal(g, 1, 64, H, d)
    k, v = normal(g, T, H, d), normal(g, T, H, d)
    slots = torch.arange(T, device=DEV) * 3
    axes = W.freq_axes(d // 2, layout)
    pos3 = torch.randint(0, 50000, (T, 3), generator=g, device=DEV)
    rope = K.Rope(1e6, d, freq_axis=axes, axis_delta=pos3)
    K.kamera_append_kv(pk, pv, k, v, rope, None, slots)
    torch.cuda.synchronize()
    inv = 1e6 ** (-2.0 * np.arange(d // 2) / d)
    x = R.f64(k)
    near(pk[0, slots], R.turned(x, pos3.cpu().numpy()[:, axes], inv, 0, False), R.turn_scale(x, d // 2, 0, False),
         layout)


def test_append_model_frequency_table():
    """A model's own frequencies, with ones above a turn a token, below zero and zero."""
    T, d = 33, 64
    g = torch.Generator(device=DEV).manual_seed(4)
    inv = np.concatenate([[0.0, 7.5, -0.3, 6.283185307179586, 1e-9, 2.5e3], W.model_inv_freq("extended", 1e4, d)[6:]])
    pk, pv = normal(g, 1, 64, 1, d), normal(g, 1, 64, 1, d)
    k, v = normal(g, T, 1, d), normal(g, T, 1, d)
    pos = torch.randint(0, 100000, (T,), generator=g, device=DEV)
    K.kamera_append_kv(pk, pv, k, v, K.Rope(1e4, d, inv_freq=inv), pos, torch.arange(T, device=DEV))
    torch.cuda.synchronize()
    x = R.f64(k)
    near(pk[0, :T], R.turned(x, pos.cpu().numpy(), inv, 0, False), R.turn_scale(x, d // 2, 0, False), "table")


def test_append_in_place_queries_of_a_fused_row():
    """q_out = q inside the fused projection's rows, beside k and v of the same rows."""
    T, H, Hq, d = 19, 2, 6, 64
    g = torch.Generator(device=DEV).manual_seed(5)
    fused = normal(g, T, (Hq + 2 * H) * d)
    again = fused.clone()
    pk, pv = normal(g, 1, 32, H, d), normal(g, 1, 32, H, d)
    pos = torch.arange(T, device=DEV) + 977
    views = lambda x: (x[:, :Hq * d].unflatten(1, (Hq, d)), x[:, Hq * d:(Hq + H) * d].unflatten(1, (H, d)),
                       x[:, (Hq + H) * d:].unflatten(1, (H, d)))
    q, k, v = views(fused)
    ref = K.kamera_append_kv(pk, pv, k, v, K.Rope(1e4, d), pos, torch.arange(T, device=DEV), q=q)
    q2, k2, v2 = views(again)
    pk2, pv2 = pk.clone(), pv.clone()
    got = K.kamera_append_kv(pk2, pv2, k2, v2, K.Rope(1e4, d), pos, torch.arange(T, device=DEV), q=q2, q_out=q2)
    torch.cuda.synchronize()
    assert got is q2 and torch.equal(q2, ref) and torch.equal(pk, pk2) and torch.equal(pv, pv2)
    assert torch.equal(again[:, Hq * d:], fused[:, Hq * d:])


def test_append_one_token_with_any_token_stride():
    """One token's rows from a matrix of odd width: its token stride, which no row uses, is no multiple of 8."""
    H, Hq, d = 2, 4, 64
    g = torch.Generator(device=DEV).manual_seed(9)
    wide = normal(g, 3, (Hq + 2 * H) * d + 3)[:1]
    view = lambda o, heads: wide.as_strided((1, heads, d), (wide.stride(0), d, 1), o * d)
    q, k, v = view(0, Hq), view(Hq, H), view(Hq + H, H)
    assert k.stride(0) % 8
    pk, pv = normal(g, 1, 8, H, d), normal(g, 1, 8, H, d)
    pos, slots = torch.tensor([77], device=DEV), torch.tensor([5], device=DEV)
    out = K.kamera_append_kv(pk, pv, k, v, K.Rope(1e4, d), pos, slots, q=q)
    torch.cuda.synchronize()
    inv = 1e4 ** (-2.0 * np.arange(d // 2) / d)
    for got, x in ((pk[0, slots], R.f64(k)), (out, R.f64(q))):
        near(got, R.turned(x, pos.cpu().numpy(), inv, 0, False), R.turn_scale(x, d // 2, 0, False), "one token")
    assert torch.equal(pv[0, slots], v)


def test_append_skips_and_reports_bad_rows():
    T, H, d = 6, 2, 64
    g = torch.Generator(device=DEV).manual_seed(6)
    pk, pv = normal(g, 1, 16, H, d), normal(g, 1, 16, H, d)
    before = pk.clone()
    k, v = normal(g, T, H, d), normal(g, T, H, d)
    slots = torch.tensor([3, 16, -2, 5, 7, -1], device=DEV)
    pos = torch.tensor([1, 2, 3, 2 ** 31, 5, 2 ** 40], device=DEV)    # the padding row's position is not looked at
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    K.kamera_append_kv(pk, pv, k, v, K.Rope(1e4, d), pos, slots, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == SLOT | DESCRIPTOR
    wrote = torch.tensor([3, 7], device=DEV)
    assert not torch.equal(pk[0, wrote], before[0, wrote])
    before[0, wrote] = pk[0, wrote]
    assert torch.equal(pk, before)
    assert torch.equal(pv[0, wrote], v[torch.tensor([0, 4], device=DEV)])


def test_append_past_32_bit_offsets():
    """Slots whose element offset passes 2^31 in a tall pool, and a layer past it."""
    H, d, S = 8, 128, 1 << 20
    pk = torch.empty(3, S, H, d, dtype=torch.bfloat16, device=DEV)    # 2^30 elements a layer
    pv = torch.empty(3, S, H, d, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(7)
    k, v = normal(g, 4, H, d), normal(g, 4, H, d)
    slots = torch.tensor([S - 1, 0, S // 2, S - 17], device=DEV)
    pos = torch.tensor([9, 8, 7, 6], device=DEV)
    K.kamera_append_kv(pk, pv, k, v, K.Rope(1e4, d), pos, slots, layer=2)
    torch.cuda.synchronize()
    x = R.f64(k)
    near(pk[2, slots], R.turned(x, pos.cpu().numpy(), 1e4 ** (-2.0 * np.arange(64) / 128), 0, False),
         R.turn_scale(x, 64, 0, False), "tall")
    assert torch.equal(pv[2, slots], v)


def test_append_captured_and_on_another_stream():
    """One captured step, replayed with new inputs in place, and one on a side stream."""
    T, H, d = 8, 2, 64
    g = torch.Generator(device=DEV).manual_seed(8)
    pk, pv = normal(g, 1, 64, H, d), normal(g, 1, 64, H, d)
    k, v, q = normal(g, T, H, d), normal(g, T, H, d), normal(g, T, 4, d)
    pos, slots = torch.arange(T, device=DEV), torch.arange(T, device=DEV) * 2
    rope = K.Rope(1e4, d)
    K.kamera_append_kv(pk, pv, k, v, rope, pos, slots, q=q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = K.kamera_append_kv(pk, pv, k, v, rope, pos, slots, q=q)
    k.copy_(normal(g, T, H, d))
    q.copy_(normal(g, T, 4, d))
    pos.add_(1000)
    slots.add_(1)
    graph.replay()
    torch.cuda.synchronize()
    pk2, pv2 = pk.clone(), pv.clone()
    pk2[0, slots] = 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2 = K.kamera_append_kv(pk2, pv2, k, v, rope, pos, slots, q=q, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(pk, pk2) and torch.equal(pv, pv2) and torch.equal(out, out2)
