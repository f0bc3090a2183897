"""Decode steps over the paged pool at their edges.  Tolerances are those of
test_gpu_append and test_gpu_paged."""
import numpy as np
import pytest
import torch

import position_invariant_kv_chunk_gb300 as K
from tests import paged_ref as R
from tests.test_gpu_paged import DEV, Pool, boxes, i32, near, normal, select_ref

pytestmark = pytest.mark.gpu


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
