"""The 4-bit cache row, the attention step and the attention-weight round from their definitions, in 64 bits (numpy),
for the tests.  Nothing here calls the library."""
import numpy as np


def code_rows(x):
    """(step, lo, codes) of rows x [..., d] float64 (each a bf16 value): step and lo [..., 4], codes [..., 4, d/4].
    A group that is not finite, or too wide, has NaN step and lo and codes 0.  Differences and quotients are rounded to
    fp32, as the definition says (numpy's float32 operations are correctly rounded)."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], 4, x.shape[-1] // 4)
    fine = np.isfinite(g).all(-1)
    safe = np.where(fine[..., None], g, 0.0).astype(np.float32)
    lo = safe.min(-1)
    with np.errstate(over="ignore"):
        r = ((safe.max(-1) - lo) / np.float32(15.0)).astype(np.float64)
    m, e = np.frexp(r)
    step = np.where(r >= 2.0 ** -56, np.ldexp(np.ceil(m * 16) / 16, e), 0.0)
    bad = ~fine | (r >= 2.0 ** 56)
    codes = np.zeros(g.shape)
    on = (step > 0) & ~bad
    codes[on] = np.rint((safe[on] - lo[on][..., None]) / step[on][..., None].astype(np.float32))
    assert codes.min(initial=0) >= 0 and codes.max(initial=0) <= 15
    return np.where(bad, np.nan, step), np.where(bad, np.nan, lo.astype(np.float64)), np.where(bad[..., None], 0.0, codes)


def centres(step, lo):
    """(z, mid) of a V row's finite groups: z = min(15, rint(-lo / step)) where 0 < -lo / 2^e < 32, mid = lo + z * step."""
    unit = np.where(step > 0, 2.0 ** (np.frexp(step)[1] - 1), 1.0)
    on = (step > 0) & (-lo / unit > 0) & (-lo / unit < 32)
    z = np.where(on, np.minimum(np.rint(np.float32(-lo) / np.where(step > 0, step, 1).astype(np.float32)), 15), 0.0)
    return z, lo + z * step


def k_order(codes):
    """Codes [..., d] of K rows in the order of the row's bytes: unit t of group g is unit 4 t + g."""
    u = codes.reshape(*codes.shape[:-1], 4, 4, codes.shape[-1] // 16)  # group, unit, channel
    return u.swapaxes(-3, -2).reshape(codes.shape)


def row_values(x):
    """The values that the coded rows stand for."""
    step, lo, codes = code_rows(x)
    return (lo[..., None] + step[..., None] * codes).reshape(np.shape(x))


def attention(q, k, v, scale):
    """One step for q [G, d] over rows k, v [L, d]: (out [G, d], lse [G], weights [L] summed over the G heads)."""
    s = scale * (q @ k.T)
    top = s.max(-1, keepdims=True)
    lse = top[:, 0] + np.log(np.exp(s - top).sum(-1))
    a = np.exp(s - lse[:, None])
    return a @ v, lse, a.sum(0)


def attention_round(weights, pos, prompt, budget, recent, next_pos):
    """Kept slots (ascending) of one segment by accumulated weight: weights and pos [L]."""
    L = len(weights)
    if L <= budget:
        return np.arange(L)
    m = max(0, budget - prompt)
    newest = next_pos - min(recent, m)

    def rank(j):
        if pos[j] >= newest:
            return (0, 0.0, pos[j])
        return (2, 0.0, pos[j]) if np.isnan(weights[j]) else (1, -weights[j], pos[j])

    best = sorted(range(prompt, L), key=rank)[:m]
    return np.array(list(range(prompt)) + sorted(best), np.int64)


def compacted(kept, new_len, hole_fill):
    """Source slot of every slot of the new cache."""
    if not hole_fill:
        return kept
    out = np.full(new_len, -1, np.int64)
    stay = kept[kept < new_len]
    out[stay] = stay
    out[np.nonzero(out < 0)[0]] = kept[kept >= new_len]
    return out
