"""Plain 64-bit forms of the decode-step operators over the paged pool, on the
CPU, token by token from their definitions.  No code of the library."""
import numpy as np
import torch


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def ulp_half(x: np.ndarray) -> np.ndarray:
    """Largest rounding of a value to bf16: half a step, 2^-8 relative."""
    return 2.0 ** -8 * np.abs(x)


def turned(x: np.ndarray, pos: np.ndarray, inv_freq: np.ndarray, off: int, interleaved: bool) -> np.ndarray:
    """R(pos) x for rows x [T, heads, width]; pos [T] or, per frequency, [T, n_freq]."""
    n = len(inv_freq)
    y = x.copy()
    for f in range(n):
        a, b = (off + 2 * f, off + 2 * f + 1) if interleaved else (off + f, off + f + n)
        p = pos if pos.ndim == 1 else pos[:, f]
        ang = (p.astype(np.float64) * inv_freq[f])[:, None]
        y[..., a] = x[..., a] * np.cos(ang) - x[..., b] * np.sin(ang)
        y[..., b] = x[..., b] * np.cos(ang) + x[..., a] * np.sin(ang)
    return y


def turn_scale(x: np.ndarray, n: int, off: int, interleaved: bool) -> np.ndarray:
    """|a| + |b| of each component's pair (0 outside the rotary range)."""
    s = np.zeros_like(x)
    for f in range(n):
        a, b = (off + 2 * f, off + 2 * f + 1) if interleaved else (off + f, off + f + n)
        s[..., a] = s[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return s


def slots_of(table, page_size: int, n: int, num_pages: int):
    """Slots of tokens 0..n-1; -1 where the page lies outside the pool."""
    out = []
    for t in range(n):
        g = int(table[t // page_size])
        out.append(g * page_size + t % page_size if 0 <= g < num_pages else -1)
    return np.array(out, dtype=np.int64)


def attention(q: np.ndarray, K: np.ndarray, V: np.ndarray, scale: float):
    """q [G, d], K and V [n, d] -> out [G, d], lse [G], and for the tolerance
    sum_j p_j |V_j| and the largest |scale| sum_i |q_i K_ji|."""
    G, d = q.shape
    if K.shape[0] == 0:
        return np.zeros((G, d)), np.full(G, -np.inf), np.zeros((G, d)), np.zeros(G)
    z = scale * (q @ K.T)
    m = z.max(1, keepdims=True)
    w = np.exp(z - m)
    l = w.sum(1, keepdims=True)
    p = w / l
    return p @ V, (m + np.log(l))[:, 0], p @ np.abs(V), abs(scale) * (np.abs(q) @ np.abs(K).T).max(1)


def page_scores(q: np.ndarray, lo: np.ndarray, hi: np.ndarray) -> np.ndarray:
    """q [G, d], boxes lo and hi [n, d] -> the bound of each page, summed over the heads."""
    return np.maximum(q[:, None] * lo[None], q[:, None] * hi[None]).sum((0, 2))


def select(scores: np.ndarray, k: int, n_first: int, n_last: int) -> list:
    n = len(scores)
    s = [float(x) for x in scores]
    for j in range(n):
        if j < n_first or j >= n - n_last or not np.isfinite(s[j]):
            s[j] = np.inf
    forced = [j for j in range(n) if j < n_first or j >= n - n_last]
    if n <= k:
        return list(range(n)) + [-1] * (k - n)
    rest = sorted((j for j in range(n) if j not in set(forced)), key=lambda j: (-s[j], j))
    return sorted(forced + rest[:k - len(forced)])
