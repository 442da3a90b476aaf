"""Scores that are not numbers, over the bf16 and fp32 caches: the step reads them the same with and without weights, with
any split of the rows, called and captured.

A head with a NaN or +infinite score has out 0, lse -infinity and adds no weight; a score of -infinity has weight 0.
Finite heads are held to attention_bounds.simt_bounds; weights add (G + 2) u of their sum with decay * w."""
import numpy as np
import pytest
import torch

from attention_bounds import U, simt_bounds, step
from test_gpu_attention_weights import dense_weights
from test_gpu_int4 import make, np64, rows

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# rows of a request and the slots of its broken rows: alone in a page, in a warp's share, in a split; the first; a page
WHERE = [(40, ()), (1, (0,)), (17, (16,)), (129, (128,)), (300, (5,)), (300, tuple(range(16, 32))), (9001, (9000,)),
         (5000, tuple(range(0, 2048))), (33, tuple(range(33))), (0, ())]


def attend(ctx, q, out, lse, accumulate, captured):
    call = lambda: ctx.decode_attention(q, out=out, lse=lse, accumulate=accumulate, decay=0.5)  # noqa: E731
    if not captured:
        call()
    else:
        if accumulate:
            held = ctx.weights.clone()
        call()  # sets the kernels up
        if accumulate:
            ctx.weights.copy_(held)
        graph = torch.cuda.CUDAGraph()
        torch.cuda.current_stream().synchronize()
        with torch.cuda.graph(graph, stream=torch.cuda.current_stream()):
            call()
        graph.replay()
        torch.cuda.current_stream().synchronize()
        del graph
    ctx.sync()


@pytest.mark.parametrize("captured", [False, True], ids=["called", "captured"])
@pytest.mark.parametrize("cache,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("G", [1, 4])
@pytest.mark.parametrize("bad", ["nan key", "inf score", "-inf score", "nan query", "nan value"])
def test_broken_rows_read_alike(bad, G, cache, d, captured):
    lens = [n for n, _ in WHERE]
    H, R = 2, len(WHERE)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ctx = make(lens, H=H, G=G, d=d, dtype=DTYPES[cache], room=20000)
        q = rows(R, 1, H * G, d, 1, dtype=ctx.dtype)[0]  # [1, R, Hq, d]
        q[..., 3] = q[..., 3].abs() + 0.5  # the channel that meets an infinity
        if bad == "nan query":
            q[0, :, H * G - 1, 7] = float("nan")
        for r, (n, broken) in enumerate(WHERE):
            if not n:
                continue
            k, v = (rows(n, 1, H, d, 10 * r + s, dtype=ctx.dtype) for s in (2, 3))
            for j in broken:
                if bad == "nan key":
                    k[0, 0, j, 1, 5] = float("nan")
                elif bad in ("inf score", "-inf score"):
                    k[0, 0, j, 1, 3] = float(bad.split()[0])
                elif bad == "nan value":
                    v[0, 0, j, 1, 9] = float("nan")
            ctx.append([r], k, v)
        w = ctx.track_weights()
        w.uniform_()
        before = dense_weights(ctx, 0, max(lens)).clone()
        outs = []
        for accumulate in (False, True):
            out = torch.full((1, R, H * G, d), 7.0, device="cuda")
            lse = torch.full((1, R, H * G), 7.0, device="cuda")
            attend(ctx, q, out, lse, accumulate, captured)
            outs.append((out, lse))
        after = np64(dense_weights(ctx, 0, max(lens)))
        kd, vd, _ = ctx.gather_dense(0, cap=max(lens))
    side.synchronize()
    scale, before = d ** -0.5, np64(before)
    for r, (n, broken) in enumerate(WHERE):
        for h in range(H):
            qq, kk, vv = np64(q[0, r, h * G:(h + 1) * G]), np64(kd[r, h, :n]), np64(vd[r, h, :n])
            o, ll, a = step(qq, kk, vv, scale)
            read = np.isfinite(ll)
            gone = sorted(set(broken)) if h == 1 else []
            if bad in ("nan key", "inf score") and gone or n == 0:
                assert not read.any()
            elif bad == "nan query" and h == 1:
                assert read.tolist() == [True] * (G - 1) + [False]
            elif bad == "-inf score" and len(gone) == n:
                assert not read.any()
            else:
                assert read.all()
            ok = np.array([j for j in range(n) if j not in set(gone)], int) if bad == "-inf score" else np.arange(n)
            bounds = None
            if n and read.any():
                fin = np.nan_to_num(vv[ok])
                bounds = simt_bounds(np.nan_to_num(qq), kk[ok], fin, scale)
            for form, (out, lse) in zip(("plain", "accumulating"), outs):
                tag = (form, bad, r, h, n)
                got, gl = np64(out[0, r, h * G:(h + 1) * G]), np64(lse[0, r, h * G:(h + 1) * G])
                assert not got[~read].any() and np.isneginf(gl[~read]).all(), tag
                if bounds is None:
                    continue
                fine = np.isfinite(vv).all(0)  # a NaN value shows in its channel
                assert np.isnan(got[read][:, ~fine]).all(), tag
                assert (np.abs(got - o) <= bounds[0])[read][:, fine].all(), tag
                assert (np.abs(gl[read] - ll[read]) <= bounds[1][read]).all(), tag
            want = 0.5 * before[r, h, :n] + a.sum(0)
            tol = (G + 2) * U * (before[r, h, :n] + a.sum(0)) + 1e-38
            if bounds is not None:
                tol = tol + (np.where(read[:, None], bounds[2], 0) * a).sum(0)
            assert (np.abs(after[r, h, :n] - want) <= tol).all(), ("weights", bad, r, h, n)
    ctx.close()


@pytest.mark.parametrize("cache", list(DTYPES))
def test_rows_of_minus_infinity_come_first(cache):
    """Whole pages of -infinity before, between and behind finite rows: they weigh nothing."""
    n, d, G = 400, 128, 2
    ctx = make([n], H=1, G=G, d=d, dtype=DTYPES[cache])
    k, v = (rows(n, 1, 1, d, s, dtype=ctx.dtype) for s in (4, 5))
    q = rows(1, 1, G, d, 6, dtype=ctx.dtype)[0]
    q[..., 3] = 1
    gone = [j for j in range(n) if j < 64 or 128 <= j < 145 or j >= 390]
    k[0, 0, gone, 0, 3] = float("-inf")
    ctx.append([0], k, v)
    w = ctx.track_weights()
    kk, vv = np64(k[0, 0, :, 0]), np64(v[0, 0, :, 0])
    o, ll, a = step(np64(q[0, 0]), kk, vv, d ** -0.5)
    ok = [j for j in range(n) if j not in set(gone)]
    to, tl, tw = simt_bounds(np64(q[0, 0]), kk[ok], vv[ok], d ** -0.5)
    for accumulate in (False, True):
        out, lse = ctx.decode_attention(q, accumulate=accumulate)
        ctx.sync()
        assert (np.abs(np64(out[0, 0]) - o) <= to).all() and (np.abs(np64(lse[0, 0]) - ll) <= tl).all()
    got = np64(dense_weights(ctx, 0, n)[0, 0])
    assert not got[gone].any()
    assert (np.abs(got - a.sum(0)) <= (tw * a).sum(0) + (G + 2) * U * a.sum(0) + 1e-38).all()
    assert w is ctx.weights
    ctx.close()
