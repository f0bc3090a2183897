"""How far a row of an attention's output may be from its definition as a whole, which
many columns know better than any one of them.  No code of the library.

A column of a long context's output is a sum with both signs, small beside sum_j p_j |v_j|:
a bound by that sum lets a whole tile of rows go missing.  The 2-norm of a row's error has
three parts.

The weights' roundings: token j adds weight p_j u_j v_j, `weight` the half step's relative
size and the u_j independent, |u_j| <= 1, u_j^2 of mean 1/3 at most (a rounding is uniform in
its step, and smaller beside a number above the step's power of two).  With a_j = weight p_j
|v_j| the square is sum a_j^2 u_j^2, of mean sum a_j^2 / 3 and standard deviation at most
0.3 sqrt(sum a_j^4) (u^4 has mean 1/5: sqrt(1/5 - 1/9)), and the products of different rows,
which are nearly orthogonal in w columns: mean 0, standard deviation sqrt(2 / w) of the mean.
Five of either deviation are allowed.

The output's rounding: the same with a_i = 2^-8 |out_i| and no products.

The rest is relative to the whole sum, and taken at its largest: 2^x (2^-21 with its fp32
argument's rounding), a score's (terms + 2) 2^-24 of its terms' magnitudes, and the fp32
sums, rounded once for 16 tokens at least (2^-23 each): n 2^-27."""
import numpy as np

from tests import paged_ref as R


def rows(q, K, V, scale):
    """q [G, d], K [n, d], V [n, w] -> per query (out, sum_j p_j^2 |v_j|^2, sum_j p_j^4 |v_j|^4,
    largest |scale| sum |q k|, n)."""
    if len(K) == 0:
        return [(np.zeros(V.shape[1]), 0.0, 0.0, 0.0, 0) for _ in q]
    z = scale * (q @ K.T)
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    size2, smax = (V ** 2).sum(1), abs(scale) * (np.abs(q) @ np.abs(K).T).max(1)
    out, two, four = p @ V, p ** 2 @ size2, p ** 4 @ size2 ** 2
    return [(out[g], two[g], four[g], smax[g], len(K)) for g in range(len(q))]


def off(out, refs, terms, weight):
    """Per row: the error's norm over what it may be."""
    ref = np.stack([r[0] for r in refs])
    two, four, smax, n = (np.array([r[i] for r in refs]) for i in range(1, 5))
    got = R.f64(out).reshape(ref.shape)
    weights = weight ** 2 * (two / 3 * (1 + 5 * np.sqrt(2 / ref.shape[1])) + 1.5 * np.sqrt(four))
    rounding = 2.0 ** -16 * ((ref ** 2).sum(1) / 3 + 1.5 * np.sqrt((ref ** 4).sum(1)))
    rest = 2.0 ** -21 + (terms + 2) * 2.0 ** -24 * smax + n * 2.0 ** -27
    may = np.sqrt(weights) + np.sqrt(rounding) + rest * (np.sqrt(two) + np.linalg.norm(ref, axis=1))
    err = np.linalg.norm(got - ref, axis=1)
    return np.where(may > 0, err / np.where(may > 0, may, 1), np.where(err == 0, 0.0, np.inf))


def near(out, refs, terms, weight, what):
    x = off(out, refs, terms, weight)
    assert np.all(x <= 1), (what, float(x.max()))   # (a NaN is not)
