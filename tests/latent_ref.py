"""Plain 64-bit forms of latent attention and of the 4-bit pages, on the CPU, from
their definitions.  No code of the library."""
import numpy as np

from tests import paged_ref as R

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def near(out, lse, refs, terms, weight, what, least=0.0):
    """Attention outputs [rows, v] and log-sum-exps [rows] against refs, per row (out,
    lse, sum_j p_j |v_j|, largest |scale| sum |q k|, tokens).  `terms`: products of a
    score; `weight`: relative error of a weight as the product takes it.

    An output is off by its rounding to bf16 (2^-8 relative) and, times sum_j p_j |v_j|,
    by the weights' errors: their rounding, 2^x (2^-21 with the fp32 argument's
    rounding), the score's (terms + 2) 2^-24 of its terms' magnitudes -- in numerator
    and denominator alike, so twice -- and the fp32 sums over n tokens (n 2^-24 each, at
    the very most).  The log-sum-exp: the score's error, the sum's and 2^-21 + 2^-22
    |lse| for 2^x, the logarithm and the rounding.

    `least`: the absolute error of a small weight, of the row's largest; a row's sixth
    entry is then sum_j |v_j|, as a weight that small counts where the others' values are
    zero (weights held as fp16 numbers 2^7 times as large: their subnormal step is 2^-24,
    so they are off by 2^-25 where the largest is 2^7 at least, 2^-32 of it)."""
    ref, rl = np.stack([r[0] for r in refs]), np.array([r[1] for r in refs])
    mag, smax, n = np.stack([r[2] for r in refs]), np.array([r[3] for r in refs]), np.array([r[4] for r in refs])
    got, gl = R.f64(out).reshape(ref.shape), R.f64(lse).reshape(-1)
    score = (terms + 2) * 2.0 ** -24 * smax
    tol = R.ulp_half(ref) + (1 + 2.0 ** -8) * 2 * (weight + 2.0 ** -21 + score + n * 2.0 ** -24)[:, None] * mag
    if least:
        tol = tol + (1 + 2.0 ** -8) * 2 * least * np.stack([r[5] for r in refs])
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.abs(got - ref)[bad].max()))
    fin = np.isfinite(rl)
    assert np.array_equal(np.isfinite(gl), fin) and np.all(gl[~fin] == -np.inf), what
    lt = score + n * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -22 * np.abs(rl)
    assert np.all(np.abs(gl[fin] - rl[fin]) <= lt[fin]), (what, float(np.abs(gl[fin] - rl[fin]).max()))


def latent_rows(q, rows, lora, scale):
    """One sequence's absorbed attention: q [Hq, W], rows [n, W] -> refs of its heads."""
    o, l, _, x = R.attention(q, rows, np.zeros((rows.shape[0], q.shape[1])), scale)
    if rows.shape[0] == 0:
        return [(np.zeros(lora), -np.inf, np.zeros(lora), 0.0, 0) for _ in q]
    z = scale * (q @ rows.T)
    p = np.exp(z - l[:, None])
    return [(p[h] @ rows[:, :lora], l[h], p[h] @ np.abs(rows[:, :lora]), x[h], rows.shape[0]) for h in range(len(q))]


def prefill_rows(q, k, v, scale, causal):
    """q [nq, dk], k [nk, dk], v [nk, dv] of one head -> refs of its queries."""
    nq, nk = len(q), len(k)
    refs = []
    for i in range(nq):
        n = max(0, min(nk, i + 1 + nk - nq)) if causal else nk
        o, l, m, x = R.attention(q[i:i + 1], k[:n], np.zeros((n, q.shape[1])), scale)
        if n == 0:
            refs.append((np.zeros(v.shape[1]), -np.inf, np.zeros(v.shape[1]), 0.0, 0))
            continue
        p = np.exp(scale * (k[:n] @ q[i]) - l[0])
        refs.append((p @ v[:n], l[0], p @ np.abs(v[:n]), x[0], n))
    return refs


# ------------------------------------------------------------ 4-bit groups --
def e4m3(x):
    """The nearest e4m3 value (even where two are as near), 448 at the most, of x >= 0."""
    x = np.minimum(x, 1e30)
    step = 2.0 ** (np.floor(np.log2(np.maximum(x, 2.0 ** -6))) - 3)
    return np.minimum(np.rint(x / step) * step, 448.0)


def packed_groups(x, unit):
    """Groups of 16 (the last axis) -> the values that 4 bits and a scale hold."""
    x = np.where(np.isnan(x), 0.0, x)
    s = e4m3(np.abs(x).max(-1) / 6 / unit)[..., None] * unit
    a = np.minimum(np.abs(x), 7 * s)[..., None]   # past the largest level: still the nearest, and differences stay exact
    far = np.abs(a - LEVELS * s[..., None])
    best = far.min(-1, keepdims=True)
    even = np.arange(8) % 2
    code = np.where(far == best, even, 2).argmin(-1)
    return np.where(x < 0, -1.0, 1.0) * LEVELS[code] * s


def packed_page(k, v, ku=1.0, vu=1.0):
    """Keys and values [P, H, d] of a page -> the values that it holds packed."""
    P, H, d = k.shape
    pk = packed_groups(k.reshape(P, H, d // 16, 16), ku).reshape(P, H, d)
    g = v.reshape(P // 16, 16, H, d).transpose(0, 2, 3, 1)
    pv = packed_groups(g, vu).transpose(0, 3, 1, 2).reshape(P, H, d)
    return pk, pv
