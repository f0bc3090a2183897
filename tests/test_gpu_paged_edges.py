"""Decode steps over the paged pool at their edges.  Tolerances are those of
test_gpu_append and test_gpu_paged."""
import numpy as np
import pytest
import torch

import position_invariant_kv_chunk_gb300 as K
from tests.test_gpu_paged import DEV, normal

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
