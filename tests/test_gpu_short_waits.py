"""A bound of nothing for the pipeline waits while every load runs: a wait that is not met
at once gives up with copies on their way.  The calls return, each CTA having waited for
its own copies and MMAs before it left, and the next call with the usual bound is right,
bit for bit.  Nothing here faults: every address stays valid, every wait is bounded."""
import pytest
import torch

import position_invariant_kv_chunk_gb300 as K
import workloads as W
from tests import test_gpu_attend as A
from tests import test_gpu_attend_mla as M
from tests import test_gpu_latent as T
from tests import test_gpu_packed as P4
from tests import test_gpu_paged as P
from tests.test_gpu_latent import LORA, TIMEOUT, gen, i32, normal

pytestmark = pytest.mark.gpu


def gives_up_then_recovers(monkeypatch, call, times=8):
    """`call(err)` -> outputs."""
    err = i32([0])
    good = [x.clone() for x in call(err)]
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    monkeypatch.setenv("KAMERA_WAIT_LIMIT_NS", "0")
    for _ in range(times):
        call(err)
    torch.cuda.synchronize()
    assert int(err.item()) in (0, TIMEOUT)
    monkeypatch.delenv("KAMERA_WAIT_LIMIT_NS")
    err.zero_()
    again = call(err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0 and all(torch.equal(a, b) for a, b in zip(good, again))


@pytest.mark.parametrize("Hq", [16, 32, 128])
def test_latent_decode(Hq, monkeypatch):
    lens = [3000, 65, 700, 0]
    pool = T.Pool(8, 300, 16)
    table = pool.table(lens)
    q = normal(pool.g, 4, Hq, T.W)
    gives_up_then_recovers(monkeypatch, lambda err: K.kamera_mla_attend_paged(pool.kv, LORA, q, 16, table, i32(lens), 3000,
                                                                              err=err))


@pytest.mark.parametrize("tokens,H", [(100, 1), (1300, 16), (20000, 3)])
def test_expansion(tokens, H, monkeypatch):
    """Two CTAs share a barrier for their halves of the weights: either may give up first."""
    g = gen(tokens)
    pool, weight = normal(g, 700, T.W), normal(g, H, 256, LORA, std=0.05)
    slots = torch.randint(0, 700, (tokens,), generator=g, device="cuda")
    gives_up_then_recovers(monkeypatch, lambda err: K.kamera_mla_expand(pool, LORA, weight, slots, err=err), 20)


@pytest.mark.parametrize("seqs,H", [(1, 2), (4, 40)])
def test_latent_prefill(seqs, H, monkeypatch):
    g = gen(12)
    qs, ks = T.starts([390] * seqs), T.starts([700] * seqs)
    q, kv, kr = normal(g, qs[-1], H, 192), normal(g, ks[-1], H, 256), normal(g, ks[-1], 64)
    gives_up_then_recovers(monkeypatch, lambda err: K.kamera_mla_prefill_attend(q, kv, kr, i32(qs), i32(ks), 390, err=err))


@pytest.mark.parametrize("G,d", [(7, 128), (12, 64)])
def test_packed_attention(G, d, monkeypatch):
    c = P4.Cache(26, [9000, 400], [20, 130], 2, d, 16)
    q = normal(c.g, 2, 2 * G, d)
    gives_up_then_recovers(monkeypatch, lambda err: K.kamera_attend_packed(*c.args(q), err=err))


@pytest.mark.parametrize("readers,d", [(2, 128), (40, 64)])
def test_shared_prefix(readers, d, monkeypatch):
    pool = P.Pool(25, 400, 16, 2, d)
    pre, own = pool.table([5000], 313), pool.table([17] * readers, 2)
    pool.poison()
    q = P.normal(pool.g, readers, 14, d)
    args = (16, i32([0, readers]), pre, i32([5000]), own, i32([17] * readers), readers, 5000, 17)
    gives_up_then_recovers(monkeypatch, lambda err: K.kamera_attend_shared(pool.k, pool.v, q, *args, err=err))


def test_reused_chunks(monkeypatch):
    a = W.make_attend(A.CASES["qwen_gqa"], "cuda")
    gives_up_then_recovers(monkeypatch, lambda err: [A.run_attend(a, err=err)])
    a = W.make_mla_attend(M.CASES["dsv2_ragged"], "cuda")
    gives_up_then_recovers(monkeypatch, lambda err: [M.run_mla(a, err=err)])


@pytest.mark.parametrize("bound", [2 ** 63, 2 ** 63 + 7, 2 ** 64 - 1])
def test_bounds_past_63_bits_are_long(bound, monkeypatch):
    lens = [3000, 65]
    pool = T.Pool(8, 300, 16)
    table = pool.table(lens)
    q = normal(pool.g, 2, 16, T.W)
    g = gen(3)
    weight, slots = normal(g, 2, 256, LORA, std=0.05), torch.arange(1000, device="cuda")
    c = P4.Cache(26, [900, 400], [20, 130], 2, 128, 16)
    qd = normal(c.g, 2, 14, 128)
    err = i32([0])

    def calls():
        out = [*K.kamera_mla_attend_paged(pool.kv, LORA, q, 16, table, i32(lens), 3000, err=err),
               *K.kamera_mla_expand(pool.kv, LORA, weight, slots, err=err), *K.kamera_attend_packed(*c.args(qd), err=err)]
        kv, kr = out[2:4]
        out += K.kamera_mla_prefill_attend(normal(gen(1), 300, 2, 192), kv, kr, i32([0, 300]), i32([0, 1000]), 300, err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        return out
    good = calls()
    monkeypatch.setenv("KAMERA_WAIT_LIMIT_NS", str(bound))
    assert all(torch.equal(a, b) for a, b in zip(good, calls()))
