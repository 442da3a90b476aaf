"""Accumulated attention weights: the step that adds them, the rounds that move them, the selector that ranks by them.

Tolerance of a step's weights: a weight exp(s - lse) is off by the relative errors of s and lse (both bounded as in
test_gpu_int4.py and test_gpu_attention.py; the larger bound of the two kernels is used for every cache) and 4 roundings;
G of them and decay * w are added in fp32: |error| <= sum_g a_g * (2 ds + 2^-18 + chain + 8u) + (G + 2) u * (w + sum a_g)."""
import numpy as np
import pytest
import torch

import rows4
from decode_kv_cache_paged_b200 import (KVC_ERR_INVALID_ARG, KVC_ERR_NAN, KVC_ERR_STATE, KVC_ERR_UNSUPPORTED,
                                        KVC_OPT_RECENT_TOKENS, KvcError, kvc_attention_options, kvc_bind_weights,
                                        kvc_decode_attention_ex)
from test_gpu_int4 import LENS, U, check_attention, fill, make, np64, rows

pytestmark = pytest.mark.gpu

CACHES = {"int4": "int4", "bf16": torch.bfloat16, "f32": torch.float32}


def dense_weights(ctx, layer, cap):
    """[R, H, cap] of one layer, by slot; NaN past the block table."""
    assert cap <= ctx.spec.max_seq_len
    bt = ctx.state_tensors()["block_table"].long()
    slots = torch.arange(cap, device=ctx.device)
    page = bt[:, slots // 16]
    w = ctx.weights[layer, page.clamp(min=0)]  # [R, cap, H, 16]
    w = w.gather(-1, (slots % 16).view(1, cap, 1, 1).expand(w.shape[0], cap, w.shape[2], 1))[..., 0]
    return torch.where((page >= 0).unsqueeze(-1), w, float("nan")).transpose(1, 2)


def check_weights(ctx, q, before, layers, scale, decay, tag=""):
    s = ctx.spec
    lens, _ = ctx.lengths()
    d, G = s.head_dim, s.num_q_heads // s.num_kv_heads
    cap = int(max(lens.max(), 1))
    for li, layer in enumerate(layers):
        k, v, _ = ctx.gather_dense(layer, cap=cap)
        got = np64(dense_weights(ctx, layer, cap))
        for r, L in enumerate(lens):
            for h in range(s.num_kv_heads if L else 0):
                qq, kk = np64(q[li, r, h * G:(h + 1) * G]), np64(k[r, h, :L])
                _, _, a = rows4.attention(qq, kk, np64(v[r, h, :L]), scale)
                lo = np.repeat(kk.reshape(L, 4, -1).min(-1), d // 4, -1)
                A = scale * (np.abs(qq) @ (np.abs(kk - lo) + np.abs(lo)).T).max()
                ss = scale * (qq @ kk.T)
                # fp32 dot products of d terms (the 4-bit cache's bound is below this one)
                ds = (d + 8) * U * A + 2 * U * (ss.max() - ss.min()) + 4 * U
                tol = a * (2 * ds + 2.0 ** -18 + (L / 16 + 64) * 2 * U + 8 * U) + (G + 2) * U * (np64(before[layer])[r, h, :L] + a)
                err = np.abs(got[r, h, :L] - (decay * np64(before[layer])[r, h, :L] + a))
                assert np.all(err <= tol + 1e-38), (tag, layer, r, h, float((err / tol).max()))


def run_step(ctx, q, layers, scale=None, decay=1.0):
    lens, _ = ctx.lengths()
    cap = int(max(lens.max(), 1))
    before = {l: dense_weights(ctx, l, cap).clone() for l in range(ctx.spec.num_layers)}
    out, lse = ctx.decode_attention(q, layer_begin=layers[0], scale=scale or 0.0, accumulate=True, decay=decay)
    ctx.sync()
    sc = scale or ctx.spec.head_dim ** -0.5
    check_attention(ctx, q, out, lse, layers, sc)
    check_weights(ctx, q, before, layers, sc, decay)
    return before


@pytest.mark.parametrize("cache", list(CACHES))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_steps_accumulate(cache, d, G):
    ctx = make(LENS, layers=2, H=2, G=G, d=d, dtype=CACHES[cache])
    fill(ctx, LENS, seed=1)
    w = ctx.track_weights()
    assert not w.any()
    run_step(ctx, rows(len(LENS), 2, 2 * G, d, 2, dtype=ctx.dtype)[0], [0, 1])
    run_step(ctx, rows(len(LENS), 2, 2 * G, d, 3, dtype=ctx.dtype)[0], [0, 1], decay=0.75)
    run_step(ctx, rows(len(LENS), 1, 2 * G, d, 4, dtype=ctx.dtype)[0], [1], scale=0.2, decay=0.0)
    ctx.close()


@pytest.mark.parametrize("cache,G,lens", [("bf16", 4, [9001, 40, 700]), ("int4", 8, [32768, 3]), ("f32", 8, [32768]),
                                          ("bf16", 8, [32768]), ("int4", 4, [2048] * 20), ("int4", 4, [32768, 20001]),
                                          ("int4", 8, [20003, 17, 19000, 0]), ("int4", 8, [20003, 17, 19000, 0] * 5),
                                          ("int4", 2, [32768] + [5, 0, 2047, 2048, 31] * 13)], ids=str)
def test_long(cache, G, lens):
    ctx = make(lens, H=2, G=G, dtype=CACHES[cache])
    fill(ctx, lens, seed=5)
    ctx.track_weights()
    run_step(ctx, rows(len(lens), 1, 2 * G, 128, 6, dtype=ctx.dtype)[0], [0])
    ctx.close()


@pytest.mark.parametrize("G,d,H", [(8, 64, 2), (8, 128, 1), (4, 64, 32)])
def test_long_layers(G, d, H):
    """Weights by a launch of their own, two layers of three in a call."""
    lens = [20501, 0, 33]
    ctx = make(lens, layers=3, H=H, G=G, d=d)
    fill(ctx, lens, seed=6)
    w = ctx.track_weights()
    w.uniform_()
    run_step(ctx, rows(len(lens), 2, H * G, d, 7)[0], [1, 2], decay=0.5)
    ctx.close()


@pytest.mark.parametrize("cache", list(CACHES))
def test_mass_and_untouched_rows(cache):
    """A step adds G to each (layer, request, KV head) in all, and writes no other entry: neither the rows past a
    request's length, nor the other layers, nor the free pages."""
    lens = [33, 0, 250, 16]
    ctx = make(lens, layers=3, H=2, G=4, dtype=CACHES[cache])
    fill(ctx, lens, seed=7)
    w = ctx.track_weights()
    w.fill_(-3.0)
    ctx.decode_attention(rows(4, 1, 8, 128, 8, dtype=ctx.dtype)[0], layer_begin=1, accumulate=True, decay=0.0)
    ctx.sync()
    assert (w[0] == -3).all() and (w[2] == -3).all()
    dense = np64(dense_weights(ctx, 1, 250))
    for r, n in enumerate(lens):
        if n:
            # n weights, each within the tolerance above; 1e-4 of the mass is far over their sum of errors
            assert np.all(np.abs(dense[r, :, :n].sum(-1) - 4) < 4e-4)
        past = dense[r, :, n:(n + 15) // 16 * 16]
        assert np.all(past == -3)
    assert int((w[1] != -3).sum()) == 2 * sum(lens)
    ctx.close()


@pytest.mark.parametrize("cache", list(CACHES))
def test_every_row_once(cache):
    """A zero query weighs every row alike: G / L each, to the rounding of lse and exp2."""
    lens = [1, 17, 500, 4096]
    ctx = make(lens, H=2, G=2, d=64, dtype=CACHES[cache])
    fill(ctx, lens, seed=9)
    ctx.track_weights()
    ctx.decode_attention(torch.zeros((1, 4, 4, 64), dtype=ctx.dtype, device="cuda"), accumulate=True)
    ctx.sync()
    dense = np64(dense_weights(ctx, 0, 4096))
    for r, n in enumerate(lens):
        assert np.all(np.abs(dense[r, :, :n] - 2 / n) <= (8 + np.log2(n)) * 2 * U * 2 / n), (cache, n)
    ctx.close()


def test_without_accumulate_nothing_is_added():
    ctx = make([100], H=2, G=4, dtype=torch.bfloat16)
    fill(ctx, [100], seed=11)
    w = ctx.track_weights()
    q = rows(1, 1, 8, 128, 12)[0]
    a = ctx.decode_attention(q)
    assert not w.any()
    ctx.untrack_weights()
    b = ctx.decode_attention(q)
    ctx.sync()
    assert torch.equal(a[0], b[0]) and ctx.weights is None
    ctx.close()


def test_the_same_step_gives_the_same_bits():
    for cache in CACHES.values():
        ctx = make([5000, 100], H=2, G=4, dtype=cache)
        fill(ctx, [5000, 100], seed=13)
        w = ctx.track_weights()
        q = rows(2, 1, 8, 128, 14, dtype=ctx.dtype)[0]
        ctx.decode_attention(q, accumulate=True)
        first = w.clone()
        w.zero_()
        ctx.decode_attention(q, accumulate=True)
        ctx.sync()
        assert torch.equal(first, w)
        ctx.close()


def test_captured_step_follows_the_cache():
    for cache in CACHES.values():
        lens = [60, 900]
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            ctx = make(lens, H=2, G=4, dtype=cache, room=3000)
            fill(ctx, lens, seed=15)
            ctx.track_weights()
            q = rows(2, 1, 8, 128, 16, dtype=ctx.dtype)[0]
            out, lse = ctx.decode_attention(q, accumulate=True)
            side.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                ctx.decode_attention(q, out=out, lse=lse, accumulate=True)
            fill(ctx, [2900, 1200], seed=17)
            lens2, _ = ctx.lengths()
            before = {0: dense_weights(ctx, 0, int(lens2.max())).clone()}
            graph.replay()
            side.synchronize()
            check_attention(ctx, q, out, lse, [0], 128 ** -0.5)
            check_weights(ctx, q, before, [0], 128 ** -0.5, 1.0)
            side.synchronize()
        ctx.close()


# ------------------------------------------------------------------ rounds --

def distinct(shape, seed, ties):
    """Weights with exact ties (multiples of 1/8) or spread."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.exp(2 * torch.randn(shape, generator=g, device="cuda"))
    return (w * 8).round() / 8 if ties else w


def snapshot(ctx, cap):
    k, v, p = zip(*(ctx.gather_dense(l, cap=cap) for l in range(ctx.spec.num_layers)))
    w = [dense_weights(ctx, l, cap).clone() for l in range(ctx.spec.num_layers)]
    return k, v, p, w


def check_round(ctx, selector, budgets, recent, next_pos, compaction="ordered", sinks=None, seed=0):
    """One round against the definition: kept positions, K, V and weights of every segment."""
    lens, prompts = ctx.lengths()
    cap = int(max(lens.max(), 1))
    k0, v0, p0, w0 = snapshot(ctx, cap)
    ctx.compress(selector, np.asarray(budgets, np.int32), seed, compaction=compaction, sink_tokens=sinks)
    ctx.sync()
    now, _ = ctx.lengths()
    k1, v1, p1, w1 = snapshot(ctx, cap)
    for r, L in enumerate(lens):
        P = int(prompts[r]) if sinks is None else min(int(prompts[r]), sinks)
        for l in range(ctx.spec.num_layers):
            for h in range(ctx.spec.num_kv_heads):
                pos = p0[l][r, h, :L].cpu().numpy()
                if selector == "attention":
                    kept = rows4.attention_round(np64(w0[l][r, h, :L]), pos, P, budgets[r], recent, next_pos[r])
                    n = len(kept)
                    src = rows4.compacted(kept, n, compaction == "hole_fill" and L > budgets[r] and budgets[r] > P)
                else:  # the position names the row
                    n = int(now[r])
                    src = np.array([{int(x): j for j, x in enumerate(pos)}[int(x)] for x in p1[l][r, h, :n].cpu().numpy()], np.int64)
                assert now[r] == n
                s = torch.as_tensor(src, device="cuda")
                for a, b in ((p0, p1), (w0, w1), (k0, k1), (v0, v1)):
                    x, y = a[l][r, h][s], b[l][r, h, :n]
                    assert torch.equal(x.nan_to_num(nan=-7.5) if x.is_floating_point() else x,
                                       y.nan_to_num(nan=-7.5) if y.is_floating_point() else y), (r, l, h)


@pytest.mark.parametrize("cache,d", [("bf16", 128), ("int4", 64), ("f32", 64)])
@pytest.mark.parametrize("compaction", ["ordered", "hole_fill"])
@pytest.mark.parametrize("ties", [False, True])
def test_attention_rounds(cache, d, compaction, ties):
    """Rounds with appends between them: prompt, sinks, recent positions, no-op and prompt-over-budget requests."""
    prompts, lens = [16, 0, 40, 5, 0, 300], [200, 77, 60, 5, 0, 700]
    ctx = make(lens, layers=2, H=2, d=d, dtype=CACHES[cache], room=96)
    for i, n in enumerate(lens):
        x = rows(n, 2, 2, d, 300 + i, dtype=ctx.dtype)
        for a, b, prot in ((0, prompts[i], True), (prompts[i], n, False)):
            if b > a:
                ctx.append([i], x[:, :, a:b].contiguous(), x[:, :, a:b].contiguous(), protect=prot)
    w = ctx.track_weights()
    next_pos = list(lens)
    for rnd, (budgets, recent, sinks) in enumerate([([120, 64, 30, 5, 3, 600], 0, None), ([100, 60, 30, 9, 3, 500], 24, None),
                                                    ([90, 10, 12, 9, 3, 290], 24, 4)]):
        w.copy_(distinct(w.shape, 20 + rnd, ties))
        ctx.set_option(KVC_OPT_RECENT_TOKENS, recent)
        check_round(ctx, "attention", budgets, recent, next_pos, compaction, sinks)
        x = rows(6 * 16, 2, 2, d, 400 + rnd, dtype=ctx.dtype).view(2, 6, 16, 2, d).transpose(0, 1).contiguous()
        ctx.append(np.arange(6), x, x)
        next_pos = [n + 16 for n in next_pos]
        dense = dense_weights(ctx, 0, ctx.spec.max_seq_len)
        now, _ = ctx.lengths()
        for r in range(6):
            assert not dense[r, :, now[r] - 16:now[r]].any()  # new rows start at 0
    ctx.close()


@pytest.mark.parametrize("compaction", ["ordered", "hole_fill"])
def test_long_segments(compaction):
    """More than 4096 candidates: the persistent form of the round, and hole filling, twice (unordered slots)."""
    lens = [9000, 5000, 8001]
    ctx = make(lens, layers=2, H=2, d=64, dtype=torch.bfloat16, room=64)
    fill(ctx, lens, seed=40)
    w = ctx.track_weights()
    ctx.set_option(KVC_OPT_RECENT_TOKENS, 300)
    for rnd, budgets in enumerate([[4000, 4900, 300], [3000, 200, 299]]):
        w.copy_(distinct(w.shape, 50 + rnd, True))
        check_round(ctx, "attention", budgets, 300, lens, compaction)
    ctx.close()


def test_persistent_form_after_hole_filling():
    """Ordered rounds over more than 4096 candidates whose slots an earlier round left out of position order."""
    lens = [9000, 7000]
    ctx = make(lens, layers=2, H=2, d=64, dtype=torch.bfloat16)
    fill(ctx, lens, seed=41)
    w = ctx.track_weights()
    ctx.set_option(KVC_OPT_RECENT_TOKENS, 50)
    for budgets, compaction in (([8000, 6000], "hole_fill"), ([4500, 5000], "ordered")):
        w.copy_(distinct(w.shape, 52, True))
        check_round(ctx, "attention", budgets, 50, lens, compaction)
    ctx.close()


@pytest.mark.parametrize("selector", ["random", "random_shared"])
def test_other_selectors_carry_the_weights(selector):
    for compaction in ("ordered", "hole_fill"):
        lens = [300, 6000]
        ctx = make(lens, layers=2, H=2, d=64, dtype=torch.bfloat16)
        fill(ctx, lens, seed=42)
        w = ctx.track_weights()
        w.copy_(distinct(w.shape, 60, False))
        check_round(ctx, selector, [100, 1500], 0, lens, compaction, seed=9)
        ctx.close()


def test_debug_scores_and_stats():
    ctx = make([100], H=2, d=64, dtype=torch.bfloat16)
    fill(ctx, [100], seed=43)
    w = ctx.track_weights()
    w.copy_(distinct(w.shape, 61, False))
    want = dense_weights(ctx, 0, 100).clone()
    dbg = torch.full((1, 1, 2, ctx.spec.max_seq_len), -1.0, device="cuda")
    st = ctx.compress("attention", np.array([40], np.int32), 0, debug_scores=dbg, stats=True)
    assert torch.equal(dbg[0, 0, :, :100], want[0])
    assert st["evicted"] == 2 * 60 and st["candidates"] == 200 and st["score_kernel"] == 0
    ctx.close()


def test_nan_weight_is_reported_and_ranks_last():
    ctx = make([64], H=1, d=64, dtype=torch.bfloat16, room=32)
    fill(ctx, [64], seed=44)
    w = ctx.track_weights()
    w.copy_(distinct(w.shape, 62, False))
    w.view(-1)[::3] = float("nan")
    want = rows4.attention_round(np64(dense_weights(ctx, 0, 64)[0, 0]), np.arange(64), 0, 50, 0, 64)
    ctx.compress("attention", np.array([50], np.int32), 0)
    with pytest.raises(KvcError) as e:
        ctx.sync()
    assert e.value.status == KVC_ERR_NAN
    ctx.sync()  # reported once
    assert ctx.gather_dense(0, cap=50)[2][0, 0].tolist() == want.tolist()
    ctx.set_option(KVC_OPT_RECENT_TOKENS, 64)
    x = rows(20, 1, 1, 64, 45)
    ctx.append([0], x, x)
    ctx.compress("attention", np.array([20], np.int32), 0)
    with pytest.raises(KvcError):
        ctx.sync()  # the NaN rows among the older 50 are ranked
    assert ctx.gather_dense(0, cap=20)[2][0, 0].tolist() == list(range(64, 84))
    ctx.close()


def test_infinite_weights_and_zero_weights():
    ctx = make([80], H=2, d=64, dtype=torch.bfloat16)
    fill(ctx, [80], seed=45)
    w = ctx.track_weights()  # all equal: the lowest positions stay
    check_round(ctx, "attention", [70], 0, [80])
    w.copy_(distinct(w.shape, 63, True))
    w.view(-1)[5::7] = float("inf")
    check_round(ctx, "attention", [20], 3, [80])
    ctx.close()


def test_negative_zero_is_zero():
    """Weights of -0 and 0 are equal scores: the lowest positions stay."""
    for n in (80, 4200):  # the one-CTA form and the persistent one
        ctx = make([n], H=2, d=64, dtype=torch.bfloat16)
        fill(ctx, [n], seed=48)
        w = ctx.track_weights()
        w.view(-1)[::2] = -0.0
        ctx.compress("attention", np.array([n // 3], np.int32), 0)
        ctx.sync()
        assert ctx.gather_dense(0, cap=n // 3)[2][0, 1].tolist() == list(range(n // 3))
        ctx.close()


def test_contexts_on_two_streams():
    """Two contexts of other sizes, their calls interleaved on two streams, give the bits of each alone."""
    sizes = [([6000, 10], 8, 128, "int4"), ([300, 257, 0], 2, 64, "int4"), ([5000], 4, 128, torch.bfloat16)]
    alone = []
    for together in (False, True):
        streams = [torch.cuda.Stream() for _ in sizes] if together else [torch.cuda.current_stream()] * len(sizes)
        ctxs, qs, got = [], [], []
        for i, (lens, G, d, dtype) in enumerate(sizes):
            with torch.cuda.stream(streams[i]):
                ctxs.append(make(lens, H=2, G=G, d=d, dtype=dtype))
                fill(ctxs[i], lens, seed=49 + i)
                ctxs[i].track_weights()
                qs.append(rows(len(lens), 1, 2 * G, d, 70 + i)[0])
        for step in range(4):
            for i, ctx in enumerate(ctxs):
                with torch.cuda.stream(streams[i]):
                    res = ctx.decode_attention(qs[i], accumulate=step % 2 == 0)
                    if step == 3:
                        got.append(res)
        for i, ctx in enumerate(ctxs):
            ctx.sync()
            got[i] = [x.clone() for x in (*got[i], *(dense_weights(ctx, 0, max(sizes[i][0]))[r, :, :n] for r, n in enumerate(sizes[i][0])))]
            torch.cuda.synchronize()
            ctx.close()
        if not together:
            alone = got
    for a, b in zip(alone, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("cache", list(CACHES))
def test_serving_loop(cache):
    """Steps, rounds and appends as a serving loop makes them: each step against the definition over the cache as it
    stands, each round against the definition over the weights as they stand."""
    lens, G, d = [90, 33, 64], 4, 128
    ctx = make(lens, layers=2, H=2, G=G, d=d, dtype=CACHES[cache], room=64)
    fill(ctx, lens, seed=46)
    ctx.track_weights()
    ctx.set_option(KVC_OPT_RECENT_TOKENS, 8)
    next_pos = list(lens)
    for t in range(3):
        for s in range(2):
            run_step(ctx, rows(3, 2, 2 * G, d, 500 + 10 * t + s, dtype=ctx.dtype)[0], [0, 1], decay=0.9)
            x = rows(3 * 5, 2, 2, d, 600 + 10 * t + s, dtype=ctx.dtype).view(2, 3, 5, 2, d).transpose(0, 1).contiguous()
            ctx.append([0, 1, 2], x, x)
            next_pos = [n + 5 for n in next_pos]
        check_round(ctx, "attention", [60, 30, 50], 8, next_pos, "hole_fill" if t == 1 else "ordered")
    ctx.close()


# ---------------------------------------------------------------- refusals --

def test_refusals():
    ctx = make([20], H=2, G=2, d=64, dtype=torch.bfloat16)
    fill(ctx, [20], seed=47)
    q = rows(1, 1, 4, 64, 1)[0]

    def status(call, *a, **k):
        with pytest.raises(KvcError) as e:
            call(*a, **k)
        return e.value.status

    assert status(ctx.decode_attention, q, accumulate=True) == KVC_ERR_STATE
    assert status(ctx.compress, "attention", np.array([4], np.int32), 0) == KVC_ERR_STATE
    w = ctx.track_weights()
    assert kvc_bind_weights(ctx.handle, w.data_ptr(), w.numel() * 4 - 4) == KVC_ERR_INVALID_ARG
    assert kvc_bind_weights(ctx.handle, w.data_ptr() + 4, w.numel() * 4) == KVC_ERR_INVALID_ARG
    host = torch.zeros(w.numel() + 64)
    assert kvc_bind_weights(ctx.handle, (host.data_ptr() + 255) // 256 * 256, w.numel() * 4) == KVC_ERR_INVALID_ARG
    for decay in (-0.1, 1.5, float("nan")):
        assert status(ctx.decode_attention, q, accumulate=True, decay=decay) == KVC_ERR_INVALID_ARG
    out = torch.zeros((1, 1, 4, 64), device="cuda")
    for bad in (kvc_attention_options(2, 1.0), kvc_attention_options(1, 1.0, (1, 0)), kvc_attention_options(1, 1.0, (0, 1))):
        assert kvc_decode_attention_ex(ctx.handle, 0, 1, q.data_ptr(), 0.0, bad, out.data_ptr(), None, None) == KVC_ERR_INVALID_ARG
    assert status(ctx.compress, "attention", np.array([4], np.int32), 0, block=4) == KVC_ERR_INVALID_ARG
    for value in (-1, 32769):
        assert status(ctx.set_option, KVC_OPT_RECENT_TOKENS, value) == KVC_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        ctx.track_weights(torch.zeros((1, 2, 3, 16), device="cuda"))
    assert not w.any()
    ctx.close()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ctx = make([20], H=2, G=2, d=64, dtype=torch.bfloat16)
        w = ctx.track_weights()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            w.add_(1)
            assert status(ctx.track_weights, w) == KVC_ERR_STATE
        side.synchronize()
        ctx.close()
    wide = make([20], H=2, G=1, d=256, dtype=torch.bfloat16)
    assert status(wide.track_weights) == KVC_ERR_UNSUPPORTED
    wide.close()
    odd = make([20], H=2, G=3, d=64, dtype=torch.bfloat16)
    odd.track_weights()
    assert status(odd.decode_attention, rows(1, 1, 6, 64, 1)[0], accumulate=True) == KVC_ERR_UNSUPPORTED
    odd.close()
