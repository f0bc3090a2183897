"""The scale of latent decode attention as a caller gives it.  Runs without a GPU."""
import pytest
import torch

import position_invariant_kv_chunk_gb300 as K


@pytest.fixture
def passed_on(monkeypatch):
    """The scales that calls hand to the binding."""
    got = []

    class Fast:
        @staticmethod
        def mla_attend_paged(*a):
            got.append(a[7])
    monkeypatch.setattr(K, "_FAST", Fast)
    return got


def test_scale_is_the_heads_or_given(passed_on):
    i32 = torch.zeros(1, 1, dtype=torch.int32)
    args = (torch.zeros(16, 576, dtype=torch.bfloat16), 512, torch.zeros(1, 2, 576, dtype=torch.bfloat16), 16, i32, i32[0], 16)
    K.kamera_mla_attend_paged(*args, nope_dim=128)
    K.kamera_mla_attend_paged(*args, scale=0.25)
    K.kamera_mla_attend_paged(*args)
    assert passed_on == [192 ** -0.5, 0.25, None]
    for bad in (dict(scale=0.1, nope_dim=128), dict(nope_dim=-1)):
        with pytest.raises(ValueError):
            K.kamera_mla_attend_paged(*args, **bad)
    with pytest.raises(TypeError):
        K.kamera_mla_attend_paged(*args, nope_dim=1.5)
