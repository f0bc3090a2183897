"""What the bounds of attention outputs let through, on results with a planted mistake.
Runs without a GPU: the results are this file's own arithmetic."""
import numpy as np
import pytest
import torch

from tests import attended_norm as N
from tests import latent_ref as L


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).double().numpy()


def attended(q, K, V, scale, weights=bf16):
    """The sum of rounded weights times values over the sum of the weights, rounded to bf16."""
    z = scale * (q @ K.T)
    p = np.exp(z - z.max(1, keepdims=True))
    return torch.from_numpy(weights(p) @ V / p.sum(1, keepdims=True)).to(torch.bfloat16)


# (tokens, query and key width, value width, tokens of a tile): decode, its longest; prefill
@pytest.mark.parametrize("n,d,w,tile", [(9000, 576, 512, 64), (40000, 576, 512, 64), (2500, 192, 128, 128), (9000, 192, 128, 128)])
@pytest.mark.parametrize("weight,rounding", [(2.0 ** -8, bf16), (2.0 ** -16, lambda p: p * (1 + 2.0 ** -17)),
                                             (2.0 ** -11, lambda p: p.astype(np.float16).astype(np.float64))])
def test_one_wrong_tile_is_seen(n, d, w, tile, weight, rounding):
    rng = np.random.default_rng(n)
    q, K = bf16(rng.standard_normal((3, d))), bf16(rng.standard_normal((n, d)))
    V = K[:, :w] if w == 512 else bf16(rng.standard_normal((n, w)))
    scale = d ** -0.5
    refs = N.rows(q, K, V, scale)
    N.near(attended(q, K, V, scale, rounding), refs, d, weight, "right")
    a, b = n // tile // 3 * tile, n // tile // 2 * tile
    gone, other = V.copy(), V.copy()
    gone[a:a + tile] = 0
    other[a:a + tile] = V[b:b + tile]
    for wrong in (gone, other):
        assert np.all(N.off(attended(q, K, wrong, scale, rounding), refs, d, weight) > 1)


def test_a_bound_by_every_terms_magnitude_lets_it_through():
    """Why the norm is looked at: the bound by sum_j p_j |v_j| alone takes a result without
    64 of 9000 tokens' values."""
    n, d, w = 9000, 576, 512
    rng = np.random.default_rng(5)
    q, K = bf16(rng.standard_normal((3, d))), bf16(rng.standard_normal((n, d)))
    gone = K[:, :w].copy()
    gone[4992:5056] = 0
    z = d ** -0.5 * (q @ K.T)
    lse = np.log(np.exp(z).sum(1))
    L.near(attended(q, K, gone, d ** -0.5), torch.from_numpy(lse), L.latent_rows(q, K, w, d ** -0.5), d, 2.0 ** -8, "gone")


def test_one_column_a_tile_shows_a_wrong_tile_to_any_bound():
    """Values that are 1 in the column of their tile alone leave nothing to cancel."""
    n, d, w = 9000, 576, 512
    rng = np.random.default_rng(6)
    q, K = bf16(rng.standard_normal((3, d))), bf16(rng.standard_normal((n, d)))
    q[:, :w] = 0
    K[:, :w] = np.arange(n)[:, None] // 64 % w == np.arange(w)
    refs = L.latent_rows(q, K, w, d ** -0.5)
    z = d ** -0.5 * (q @ K.T)
    lse = torch.from_numpy(np.log(np.exp(z).sum(1)))
    L.near(attended(q, K, K[:, :w], d ** -0.5), lse, refs, d, 2.0 ** -8, "right")
    gone = K[:, :w].copy()
    gone[4992:5056] = 0
    with pytest.raises(AssertionError):
        L.near(attended(q, K, gone, d ** -0.5), lse, refs, d, 2.0 ** -8, "gone")
