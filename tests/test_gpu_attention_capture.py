"""Captured decode steps: planned for every length that a replay may meet, made of kernels that the call before the capture
has loaded, and as fast as the same step called."""
import json
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from decode_kv_cache_paged_b200 import Context, ContextSpec
from test_gpu_attention_weights import CACHES, check_weights, dense_weights
from test_gpu_int4 import check_attention, fill, make, rows

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


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


@pytest.mark.parametrize("accumulate", [False, True], ids=["step", "weights"])
def test_many_units_captured_over_an_empty_cache(accumulate):
    """Units enough for the form with one warp a unit, captured before any row is there."""
    R, layers, H, G, d = 64, 7, 8, 2, 64
    then = [(37 * i) % 900 for i in range(R - 1)] + [6000]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ctx = Context(ContextSpec(num_requests=R, num_layers=layers, num_kv_heads=H, head_dim=d, max_seq_len=32768,
                                  num_pages=4096, num_q_heads=H * G), dtype="int4")
        if accumulate:
            ctx.track_weights()
        q = rows(R, layers, H * G, d, 41, dtype=ctx.dtype)[0]
        out, lse = ctx.decode_attention(q, accumulate=accumulate)
        side.synchronize()
        assert not out.any() and torch.isneginf(lse).all()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            ctx.decode_attention(q, out=out, lse=lse, accumulate=accumulate)
        fill(ctx, then, seed=42)
        graph.replay()
        side.synchronize()
        for layer in (0, layers - 1):
            check_attention(ctx, q[layer:layer + 1], out[layer:layer + 1], lse[layer:layer + 1], [layer], d ** -0.5)
            if accumulate:
                none = {layer: torch.zeros((R, H, max(then)), device="cuda")}
                check_weights(ctx, q[layer:layer + 1], none, [layer], d ** -0.5, 1.0)
        side.synchronize()
        del graph
    ctx.close()


# One short call, then a capture whose longest rows may be 32768, in a process that has loaded nothing before.  Prints the
# kernels of the capture and those of them that the call had not loaded, and the largest difference from a call's outputs.
FRESH = r"""
import json, sys
sys.path[:0] = {paths!r}
import torch
from cuda.bindings import driver as cu
from decode_kv_cache_paged_b200 import Context, ContextSpec

def ok(res):
    assert res[0] == cu.CUresult.CUDA_SUCCESS, res
    return res[1] if len(res) == 2 else res[1:]

def functions(graph):
    # the graph's kernel nodes
    n = ok(cu.cuGraphGetNodes(graph, 0))[1]
    for node in ok(cu.cuGraphGetNodes(graph, n))[0]:
        if ok(cu.cuGraphNodeGetType(node)) == cu.CUgraphNodeType.CU_GRAPH_NODE_TYPE_KERNEL:
            p = ok(cu.cuGraphKernelNodeGetParams(node))
            yield p.func if int(p.func) else ok(cu.cuKernelGetFunction(p.kern))

def name(f):
    return ok(cu.cuFuncGetName(f)).decode()

def capture(ctx, q, out, lse, acc):
    s = side.cuda_stream
    ok2 = cu.cuStreamBeginCapture(s, cu.CUstreamCaptureMode.CU_STREAM_CAPTURE_MODE_THREAD_LOCAL)
    assert ok2[0] == cu.CUresult.CUDA_SUCCESS
    ctx.decode_attention(q, out=out, lse=lse, accumulate=acc)
    return ok(cu.cuStreamEndCapture(s))

cache, d, G, R, longest, H, warm = {case!r}
dtype = "int4" if cache == "int4" else getattr(torch, cache)
side = torch.cuda.Stream()
with torch.cuda.stream(side):
    def context(max_len, dtype=dtype, d=d, G=G, R=R, H=H):
        ctx = Context(ContextSpec(num_requests=R, num_layers=1, num_kv_heads=H, head_dim=d, max_seq_len=max_len,
                                  num_pages=max(R * 8, max_len // 16), num_q_heads=H * G), dtype=dtype)
        x = torch.randn((R, 1, 100, H, d), device="cuda").to(ctx.dtype)
        ctx.append(list(range(R)), x, x)
        return ctx
    # the modules of the attention kernels: of a step over another cache, and of the call before the capture
    modules = dict()
    def step_of(ctx, acc):
        q = torch.randn((1, ctx.spec.num_requests, ctx.num_q_heads, ctx.spec.head_dim), device="cuda").to(ctx.dtype)
        out, lse = ctx.decode_attention(q, accumulate=acc)
        side.synchronize()
        for f in functions(capture(ctx, q, out, lse, acc)):
            module = ok(cu.cuFuncGetModule(f))
            modules[int(module)] = module
        return q, out, lse
    step_of(context(128, torch.bfloat16, 64, 1, 1, 1), False)
    small = context(128)
    small.track_weights()
    q, out, lse = step_of(small, warm)
    loaded = set()
    for m in modules.values():
        n = ok(cu.cuModuleGetFunctionCount(m))
        for f in ok(cu.cuModuleEnumerateFunctions(n, m)):
            if ok(cu.cuFuncIsLoaded(f)) == cu.CUfunctionLoadingState.CU_FUNCTION_LOADING_STATE_LOADED:
                loaded.add(name(f))
    big = context(longest)
    big.track_weights()
    used, apart = [], 0.0
    for acc in (False, True):
        o, l = torch.zeros_like(out), torch.zeros_like(lse)
        graph = capture(big, q, o, l, acc)
        used += [name(f) for f in functions(graph)]
        run = ok(cu.cuGraphInstantiate(graph, 0))
        assert cu.cuGraphLaunch(run, side.cuda_stream)[0] == cu.CUresult.CUDA_SUCCESS
        side.synchronize()
        w, _ = big.decode_attention(q, accumulate=acc)
        side.synchronize()
        apart = max(apart, float((o - w).abs().max()))
    small.sync(); big.sync()
print(json.dumps(dict(used=used, missing=[k for k in used if k not in loaded], apart=apart, top=float(w.abs().max()))))
"""


@pytest.mark.parametrize("case", [("int4", 128, 4, 2, 32768, 2, False), ("int4", 128, 8, 70, 32768, 8, False),
                                  ("int4", 64, 4, 2, 32768, 2, True), ("bfloat16", 128, 4, 2, 32768, 2, False),
                                  ("float32", 64, 2, 3, 32768, 2, True)], ids=str)
def test_a_capture_meets_no_kernel_that_the_call_left_unloaded(case):
    code = FRESH.format(paths=[os.path.dirname(HERE)], case=case)
    env = dict(os.environ, CUDA_MODULE_LOADING="LAZY")
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, env=env)
    assert run.returncode == 0, run.stderr[-3000:]
    got = json.loads(run.stdout.splitlines()[-1])
    print(got)
    assert got["used"] and not got["missing"]
    assert got["apart"] <= 1e-5 * got["top"]
