"""Error bounds of decode attention in fp32, for the tests, and a step from its definition in 64 bits.  Numpy only."""
import numpy as np

U = 2.0 ** -24
LAM = 8.0  # of the probabilistic rounding-error model (Higham and Mary, SIAM J. Sci. Comput. 2019)


def step(q, k, v, scale):
    """out [G, d], lse [G] and weights [G, L] of one step for q [G, d] over rows k, v [L, d].  A score of -infinity has
    weight 0; a head without a finite score, or with a NaN or +infinite one, has out 0, lse -infinity and weights 0."""
    with np.errstate(invalid="ignore", over="ignore"):
        s = scale * (q @ k.T)
        top = s.max(-1, initial=-np.inf)
        read = np.isfinite(top) & ~np.isnan(s).any(-1)
        p = np.where(read[:, None], np.exp(s - np.where(read, top, 0)[:, None]), 0.0)
        total = p.sum(-1)
        a = p / np.where(read, total, 1)[:, None]
        lse = np.where(read, top + np.log(np.where(read, total, 1)), -np.inf)
        out = np.where(read[:, None], a @ np.where(np.isfinite(v), v, 0.0), 0.0)
    return out, lse, a


def simt_bounds(q, k, v, scale):
    """(out [G, d], lse [G], relative weight [G, 1]) bounds of the bf16 and fp32 kernels over finite rows k, v [L, d]: scores
    of d rounded terms, sums of L terms and some 64 merges."""
    d, L = k.shape[1], k.shape[0]
    s = scale * (q @ k.T)
    A = (scale * (np.abs(q) @ np.abs(k).T)).max(-1)
    ds = LAM * np.sqrt(d + 6) * U * A + U * (s.max(-1) - s.min(-1)) + 3 * U
    acc = LAM * np.sqrt(L + 64) * U
    lse = s.max(-1) + np.log(np.exp(s - s.max(-1, keepdims=True)).sum(-1))
    dl = ds + acc + 4 * U * np.abs(lse)
    return np.abs(v).max(0) * (2 * ds + 2 * acc)[:, None] + 1e-30, dl, (ds + dl + 8 * U)[:, None]


# ---- the 4-bit cache, on inputs whose coded values and scores leave it few roundings --

GRID_SCALE = 2.0 ** -4


def grid_rows(rng, n, d, low, unit):
    """n rows [n, d] whose groups of d/4 channels hold unit * (code + low), codes of 0 to 15 with both ends in each group:
    their 4-bit form is exact, with step = unit (a power of two)."""
    c = rng.integers(0, 16, (n, 4, d // 4)).astype(np.float64)
    first = rng.integers(0, d // 4, (n, 4, 1))
    np.put_along_axis(c, first, 0.0, -1)
    np.put_along_axis(c, (first + 1 + rng.integers(0, d // 4 - 1, first.shape)) % (d // 4), 15.0, -1)
    return unit * (c.reshape(n, d) + low)


def grid_case(rng, n, d, G):
    """q [G, d], k and v [n, d] of bf16 values.  Keys k >= 0 with lo = 0; values around 0 with mid = 0; queries of 16
    channels over ten binades."""
    q = np.zeros((G, d))
    for g in range(G):
        at = rng.permutation(d)[:16]
        e = np.concatenate([[0], rng.integers(0, 10, 15)])
        q[g, at] = rng.choice([-1, 1], 16) * (128 + rng.integers(0, 128, 16)) / 128 * 2.0 ** -e
    return q, grid_rows(rng, n, d, 0, 2.0 ** -3), grid_rows(rng, n, d, -8, 2.0 ** -2)


def int4_grid_bounds(q, k, v, scale=GRID_SCALE):
    """(out, lse, weights [G, n]) bounds for grid_case inputs of at most 16 rows.

    Scores: the products of codes and the query's two parts, and their sums within a group, are exact (8 query heads: the
    remainder's products join the integers' sums and may lose 2u each); s joins the groups in up to 8 fp32 roundings, and
    log2(e), the scaling and the subtraction of the maximum add one each: 20 u A_j with A_j = scale sum_i |q_i| k_ji.
    ex2.approx is off by at most 2^-22 = 4u.  To first order an error e_j of ln p_j moves out by sum_j a_j (v_j - out) e_j.
    Second product: P's three terms hold its 24 bits; v has 4 bits and a sign, so the first two terms' products and sums fit
    24 bits and the third's sum loses at most 2u of it, in the output's sum and in the softmax's; seven fp32 roundings follow."""
    o, lse, a = step(q, k, v, scale)
    e = 20 * U * scale * (np.abs(q) @ k.T) + 4 * U  # [G, n]
    more = 1 + 2.0 ** -10  # what is left of higher order
    out = np.einsum("gn,gnd->gd", a * e, np.abs(v[None] - o[:, None])) + 4 * U * (a @ np.abs(v)) + 7 * U * np.abs(o)
    d_lse = (a * e).sum(-1) + 2 * U + 4 * U * (1 + np.abs(lse))
    return out * more, d_lse * more, a * (e + d_lse[:, None] + 6 * U) * more
