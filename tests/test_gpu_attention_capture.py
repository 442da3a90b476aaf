"""Captured decode steps: planned for every length that a replay may meet, and as fast as the same step called."""
import numpy as np
import pytest
import torch

from decode_kv_cache_paged_b200 import Context, ContextSpec
from test_gpu_attention_weights import CACHES, check_weights, dense_weights
from test_gpu_int4 import check_attention, fill, make, rows

pytestmark = pytest.mark.gpu


def timed_us(ctx, q, accumulate, captured, steps=8, repeats=7):
    """Device time of one step, the least of some repeats: `steps` calls, or as many captured ones, between two events."""
    stream = torch.cuda.current_stream()
    out, lse = ctx.decode_attention(q, accumulate=accumulate)

    def loop():
        for _ in range(steps):
            ctx.decode_attention(q, out=out, lse=lse, accumulate=accumulate)

    loop()
    if captured:
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            loop()
        loop = graph.replay
        loop()
    best = float("inf")
    for _ in range(repeats):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        loop()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 1000 / steps)
    stream.synchronize()
    return best


# cache, requests, layers, KV heads, query heads a KV head, rows, whether the step accumulates, and how many times the call's
# time it may take (with weights it keeps shared memory for the scores of the longest rows)
SERVED = [("bf16", 1, 1, 8, 4, 2048, False, 1.5), ("f32", 1, 1, 2, 4, 2048, False, 1.5), ("bf16", 4, 1, 2, 4, 4096, False, 1.5),
          ("int4", 128, 4, 8, 4, 2048, False, 1.5), ("int4", 64, 8, 8, 8, 2048, False, 1.5), ("int4", 64, 1, 8, 8, 2048, False, 1.5),
          ("int4", 1, 1, 8, 4, 2048, False, 1.5), ("int4", 128, 2, 8, 4, 2048, True, 1.5), ("bf16", 128, 1, 8, 4, 2048, True, 3.0)]


@pytest.mark.parametrize("cache,R,layers,H,G,n,accumulate,times", SERVED)
def test_a_captured_step_costs_what_the_call_does(cache, R, layers, H, G, n, accumulate, times):
    """Rows far below the context's maximum, which a replay may reach: a multiple of the call's time, and 5 us, are allowed."""
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ctx = Context(ContextSpec(num_requests=R, num_layers=layers, num_kv_heads=H, head_dim=128, max_seq_len=32768,
                                  num_pages=max(R * n // 16, 2048), num_q_heads=H * G), dtype=CACHES[cache])
        for r in range(R):
            x = rows(n, layers, H, 128, r, dtype=ctx.dtype)
            ctx.append([r], x, x)
        if accumulate:
            ctx.track_weights()
        q = rows(R, layers, H * G, 128, 77, dtype=ctx.dtype)[0]
        called = timed_us(ctx, q, accumulate, False)
        captured = timed_us(ctx, q, accumulate, True)
        print(f"called {called:.1f} us, captured {captured:.1f} us")
        assert captured <= times * called + 5
        ctx.sync()
    ctx.close()


@pytest.mark.parametrize("accumulate", [False, True], ids=["step", "weights"])
@pytest.mark.parametrize("cache", list(CACHES))
@pytest.mark.parametrize("first,then", [([0, 0, 0], [3, 9001, 20000]), ([20, 300, 5], [40, 350, 4099]),
                                        ([9001, 16, 0], [20011, 17, 1])], ids=str)
def test_replays_follow_the_lengths(first, then, cache, accumulate):
    """Captured over short, middling and long rows, replayed over longer ones, then over the rows that a round left."""
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ctx = make([0, 0, 0], H=2, G=4, dtype=CACHES[cache], room=20032)
        fill(ctx, first, seed=31)
        if accumulate:
            ctx.track_weights()
        q = rows(3, 1, 8, 128, 32, dtype=ctx.dtype)[0]
        out, lse = ctx.decode_attention(q, accumulate=accumulate)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            ctx.decode_attention(q, out=out, lse=lse, accumulate=accumulate)
        fill(ctx, [b - a for a, b in zip(first, then)], seed=33)
        for budgets in (None, [2, 300, 600]):
            if budgets:
                ctx.compress("random", np.array(budgets, np.int32), 4)
            q.copy_(rows(3, 1, 8, 128, 34, dtype=ctx.dtype)[0])
            lens, _ = ctx.lengths()
            before = {0: dense_weights(ctx, 0, int(lens.max())).clone()} if accumulate else None
            graph.replay()
            side.synchronize()
            check_attention(ctx, q, out, lse, [0], 128 ** -0.5)
            if accumulate:
                check_weights(ctx, q, before, [0], 128 ** -0.5, 1.0)
        side.synchronize()
        del graph
    ctx.close()
