"""Calls of latent attention and of the packed pages at the edges of what they take."""
import numpy as np
import pytest
import torch

import position_invariant_kv_chunk_gb300 as K
from tests import latent_ref as L
from tests import test_gpu_latent as T
from tests import test_gpu_packed as P4
from tests.test_gpu_latent import DESCRIPTOR, DEV, LEN, gen, i32, normal

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("qs,ks,bit", [([0, 20, 60], [0, 30, 80], LEN), ([0, 0, 60], [0, 30, 80], LEN),
                                       ([0, 0, 0], [0, 30, 80], 0), ([0, 61, 61], [0, 30, 80], DESCRIPTOR),
                                       ([0, 0, 5], [0, 81, 80], DESCRIPTOR), ([0, 0, 5], [-1, 30, 80], DESCRIPTOR | LEN)])
def test_prefill_with_a_bound_of_no_queries(qs, ks, bit):
    """A sequence with more queries than max_q is reported where max_q is 0 too."""
    g = gen(5)
    q, kv, kr = normal(g, 60, 2, 192), normal(g, 80, 2, 256), normal(g, 80, 64)
    out, lse, err = torch.full((60, 2, 128), 5.0, dtype=BF, device=DEV), torch.full((60, 2), 5.0, device=DEV), i32([0])
    K.kamera_mla_prefill_attend(q, kv, kr, i32(qs), i32(ks), 0, out=out, lse=lse, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == bit and bool((out == 5).all()) and bool((lse == 5).all())


@pytest.mark.parametrize("H,G,d", [(2, 7, 128), (1, 12, 64)])
def test_packed_attention_with_a_bound_of_no_tokens(H, G, d):
    """Lengths behind a bound of 0 are reported, in either part (max_tail is 0 where a call
    does not give it), and their tokens left out; lengths of 0 are fine, and so are none."""
    c = P4.Cache(41, [130, 0, 16], [5, 0, 20], H, d, 16)
    q = normal(c.g, 3, H * G, d)
    packed, _, P, table, lens, top, tk, tv, tt, tl, most, TP = c.args(q)
    zero, err = i32([0, 0, 0]), i32([0])

    def call(*part, **tail):
        err.zero_()
        out = K.kamera_attend_packed(packed, q, P, *part, **tail, tail_page_size=TP, err=err)
        torch.cuda.synchronize()
        return out, int(err.item())
    tail = dict(pool_k=tk, pool_v=tv, tail_pages=tt, tail_lens=tl, max_tail=most)
    no_tail = {**tail, "tail_lens": zero, "max_tail": 0}
    alone, bits = call(table, lens, top)
    assert bits == 0
    for part, kw, ref, bit in (((table, lens, top), {**tail, "max_tail": 0}, alone, LEN), ((table, lens, top), no_tail, alone, 0),
                               ((table, lens, 0), {}, None, LEN), ((table, zero, 0), {}, None, 0), ((None, None, 0), {}, None, 0),
                               ((table, lens, 0), no_tail, None, LEN), ((None, None, 0), {**tail, "max_tail": 0}, None, LEN)):
        (out, lse), bits = call(*part, **kw)
        assert bits == bit, (part[2], kw.get("max_tail"))
        if ref is None:
            assert not bool(out.any()) and bool((lse == -float("inf")).all())
        else:
            assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
    (out, lse), bits = call(table, lens, 0, **tail)                    # the tails alone
    assert bits == LEN
    (want, wl), bits = call(None, None, 0, **tail)
    assert bits == 0 and torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("Hq,nope", [(16, 128), (40, 128), (4, 0)])
def test_decode_scaled_for_the_heads_before_the_absorption(Hq, nope):
    """nope_dim gives the scale of the expanded heads' keys, the one that prefill takes."""
    lens = [200, 0, 65]
    pool = T.Pool(Hq, 30, 16)
    table = pool.table(lens)
    q = normal(pool.g, 3, Hq, T.W)
    args = (pool.kv, T.LORA, q, 16, table, i32(lens), 200)
    scale = float(np.float32((nope + 64) ** -0.5))
    out, lse = K.kamera_mla_attend_paged(*args, nope_dim=nope)
    same, sl = K.kamera_mla_attend_paged(*args, scale=(nope + 64) ** -0.5)
    torch.cuda.synchronize()
    assert torch.equal(out, same) and torch.equal(lse, sl)
    L.near(out, lse, T.decode_refs(q, pool, table, lens, scale), T.W, T.weight_error(Hq), (Hq, nope))
