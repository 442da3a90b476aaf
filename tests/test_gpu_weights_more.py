"""Tracked weights beside the beacon selectors, and seeded configurations of the 4-bit cache and of accumulating steps: the
shapes that choose between forms of the launch are drawn, not picked."""
import random

import numpy as np
import pytest
import torch

from decode_kv_cache_paged_b200 import KVC_OPT_RECENT_TOKENS, Context, ContextSpec
from test_gpu_attention_weights import CACHES, check_round, distinct, run_step
from test_gpu_int4 import fill, make, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("compaction", ["ordered", "hole_fill"])
@pytest.mark.parametrize("selector", ["beacon", "beacon_trigger"])
def test_beacon_selectors_carry_the_weights(selector, compaction):
    lens = [300, 77, 5200]
    ctx = Context(ContextSpec(num_requests=3, num_layers=2, num_kv_heads=2, head_dim=64, max_seq_len=5216, num_pages=360,
                              num_q_heads=4, num_beacons=8, query_window=16))
    for i, n in enumerate(lens):
        k, v = (rows(n, 2, 2, 64, 7 * i + s) for s in (1, 2))
        ctx.append([i], k, v, rows(n, 2, 4, 64, 7 * i + 3))
    ctx.update_beacons()
    w = ctx.track_weights()
    w.copy_(distinct(w.shape, 70, False))
    check_round(ctx, selector, [100, 64, 1500], 0, lens, compaction)
    w.copy_(distinct(w.shape, 71, False))
    check_round(ctx, selector, [50, 64, 700], 0, lens, compaction)
    ctx.close()


@pytest.mark.parametrize("seed", range(16))
def test_seeded_loops(seed):
    """Steps with and without weights, rounds and appends over a drawn configuration."""
    rng = random.Random(900 + seed)
    cache = rng.choice(["int4", "int4", "bf16", "f32"])
    d, G, H, layers = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 8]), rng.randint(1, 3)
    R = rng.choice([1, 2, 5, 17, 70])
    top = rng.choice([40, 600, 3000, 17000]) if R <= 5 else rng.choice([40, 300])
    lens = [rng.choice([0, 1, rng.randint(1, top), top]) for _ in range(R)]
    lens[rng.randrange(R)] = top
    ctx = make(lens, layers=layers, H=H, G=G, d=d, dtype=CACHES[cache], room=rng.choice([64, 20000 if R <= 5 else 64]))
    fill(ctx, lens, seed=seed)
    ctx.track_weights()
    recent = rng.choice([0, 1, 20])
    ctx.set_option(KVC_OPT_RECENT_TOKENS, recent)
    next_pos = list(lens)
    for t in range(2):
        first = rng.randrange(layers)
        which = list(range(first, rng.randint(first + 1, layers)))
        run_step(ctx, rows(R, len(which), H * G, d, 40 * seed + t, dtype=ctx.dtype)[0], which, decay=rng.choice([0.0, 0.5, 1.0]))
        now, _ = ctx.lengths()
        budgets = [max(1, rng.choice([n // 2, n - 1, n + 5])) for n in now]
        # slots out of position order only at the end: check_round ranks by position either way
        check_round(ctx, "attention", budgets, recent, next_pos, "hole_fill" if t else "ordered")
        n_new = rng.choice([1, 17])
        x = rows(R * n_new, layers, H, d, 50 * seed + t, dtype=ctx.dtype).view(layers, R, n_new, H, d).transpose(0, 1).contiguous()
        ctx.append(np.arange(R), x, x)
        next_pos = [n + n_new for n in next_pos]
    run_step(ctx, rows(R, layers, H * G, d, 60 * seed, dtype=ctx.dtype)[0], list(range(layers)))
    assert isinstance(ctx.weights, torch.Tensor)
    ctx.close()


def test_decay_is_ignored_without_accumulate():
    """As the header says: any decay, a NaN among them, beside accumulate = 0."""
    ctx = make([40], H=2, G=2, d=64)
    fill(ctx, [40], seed=1)
    q = rows(1, 1, 4, 64, 2)[0]
    want = ctx.decode_attention(q)
    for decay in (-1.0, 7.0, float("nan"), float("inf")):
        got = ctx.decode_attention(q, decay=decay)
        ctx.sync()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ctx.close()
