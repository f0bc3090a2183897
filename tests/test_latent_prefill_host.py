"""Argument checks of latent prefill at the largest counts.  No call here launches a kernel."""
import ctypes as C

import pytest

import position_invariant_kv_chunk_gb300 as K

GB = 1 << 30


@pytest.mark.parametrize("inside", ["q_start", "kv_start"])
def test_outputs_inside_the_longest_lists_are_refused(inside):
    """2^31 - 1 sequences: their starts take 8 GB."""
    at = dict(q=1 * GB, kv=2 * GB, k_rope=3 * GB, out=4 * GB, lse=5 * GB, q_start=8 * GB, kv_start=24 * GB)
    at["out"] = at[inside] + 6 * GB
    x = K._MlaPrefill(*[{**at, **dict(q_stride=192, q_head_stride=192, kv_stride=256, k_rope_stride=64, n_q=100, n_kv=300,
                                      n_seqs=2 ** 31 - 1, num_heads=1, nope_dim=128, rope_dim=64, v_dim=128, max_q=1, causal=1,
                                      scale=0.1)}[f] for f, _ in K._MlaPrefill._fields_])
    assert K.load_library().kamera_mla_prefill_attend(C.byref(x), None, None) == 1
