"""Calls of latent attention and of the packed pages at the edges of what they take."""
import numpy as np
import pytest
import torch

import position_invariant_kv_chunk_gb300 as K
from tests import latent_ref as L
from tests import test_gpu_latent as T
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
