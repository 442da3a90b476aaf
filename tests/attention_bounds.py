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
