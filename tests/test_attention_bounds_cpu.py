"""The bounds that the 4-bit attention's precision tests assert are tight enough to fail for a kernel that leaves something
out: terms of P, the query's remainder, rows.  Each mutant is computed in 64 bits but for what it drops."""
import numpy as np
import pytest

import rows4
from attention_bounds import GRID_SCALE, U, grid_case, int4_grid_bounds, step

LENGTHS = (2, 3, 5, 9, 16)


def bf16(x):
    """x (32-bit values) rounded to bf16."""
    b = np.asarray(x, np.float32).view(np.uint32)
    return ((b + 0x7FFF + (b >> 16 & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32).astype(np.float64)


def mutant(q, k, v, terms=3, remainder=True):
    """One step with P cut to its first bf16 terms, and without the remainder of the scaled query."""
    if not remainder:
        sigma = 2.0 ** (10 - np.floor(np.log2(np.abs(q).max(-1, keepdims=True))))
        q = np.rint(q * sigma) / sigma
    s = GRID_SCALE * (q @ k.T)
    top = s.max(-1, keepdims=True)
    p = np.exp(s - top).astype(np.float32).astype(np.float64)
    if terms < 3:
        cut = bf16(p)
        if terms == 2:
            cut = cut + bf16(p - cut)
        p = cut
    total = p.sum(-1, keepdims=True)
    return (p / total) @ v, (top + np.log(total))[:, 0], p / total


def worst(d, **drop):
    """Largest error in units of the bounds: outputs, lse, weights."""
    rng = np.random.default_rng(7 + d)
    at = np.zeros(3)
    for n in LENGTHS:
        for _ in range(40):
            q, k, v = grid_case(rng, n, d, 4)
            assert np.array_equal(rows4.row_values(k), k) and np.array_equal(rows4.row_values(v), v)
            st, lo, _ = rows4.code_rows(v)
            assert not rows4.centres(st, lo)[1].any()  # mid = 0
            want, bound, got = step(q, k, v, GRID_SCALE), int4_grid_bounds(q, k, v), mutant(q, k, v, **drop)
            at = np.maximum(at, [float((np.abs(g - w) / (b + 1e-300)).max()) for g, w, b in zip(got, want, bound)])
    return at


@pytest.mark.parametrize("d", [64, 128])
def test_bounds_leave_room_for_the_whole_step(d):
    assert worst(d).max() < 0.25


@pytest.mark.parametrize("d", [64, 128])
def test_dropped_terms_exceed_the_bounds(d):
    assert worst(d, terms=2)[0] > 2
    assert worst(d, terms=1)[0] > 100
    assert (worst(d, remainder=False) > 20).all()


def test_left_out_rows_exceed_the_mean_bounds():
    """The zero-query tests hold out, a mean of whole numbers, to 6 u: one row of 32768 is more."""
    v = np.random.default_rng(3).integers(0, 16, (32768, 128)).astype(np.float64)
    full = v.mean(0)
    for part in (v[:-1], v[:-2048]):
        assert (np.abs(part.mean(0) - full) > 6 * U * full).all()
