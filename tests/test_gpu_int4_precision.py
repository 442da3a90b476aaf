"""Decode attention over the 4-bit cache held to what it is built for: every bit of P, of the query and of the codes.

Inputs whose coded values are exact and whose scores round little (attention_bounds.grid_case) leave bounds that a step
without P's third term, or without the query's remainder, exceeds (test_attention_bounds_cpu.py).  Short requests are checked
beside long ones that choose the form of the launch; the long ones are checked with a zero query, whose outputs are means of
whole numbers: every sum is exact in fp32 (below 2^24), and factors, divisions and merges leave 6 u of a mean."""
import numpy as np
import pytest
import torch

from attention_bounds import GRID_SCALE, U, grid_case, grid_rows, int4_grid_bounds, step
from test_gpu_attention_weights import dense_weights
from test_gpu_int4 import make, np64

pytestmark = pytest.mark.gpu

SHORT = [2, 3, 5, 9, 16, 2, 3]

# lengths beside the short ones, layers, KV heads: forms of the launch (csrc/decode_attention4.cu)
FORMS = {"4 warps": ([], 1, 2), "8 warps, split": ([4200], 1, 2), "one warp": ([70] * 57, 7, 8),
         "clusters": ([9000, 300], 1, 8), "waves, split": ([9000, 0, 5000, 8000, 7000, 9001], 2, 8),
         "weights apart": ([20003], 1, 2)}


def dev(x, dtype=torch.bfloat16):
    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda", torch.float32).to(dtype)


@pytest.mark.parametrize("accumulate", [False, True], ids=["step", "weights"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("form", list(FORMS))
def test_short_rows_to_the_last_bits(form, G, d, accumulate):
    more, layers, H = FORMS[form]
    lens = SHORT + more
    R = len(lens)
    ctx = make(lens, layers=layers, H=H, G=G, d=d)
    rng = np.random.default_rng(100 * G + d)
    q = np.zeros((layers, R, H * G, d))
    given = []
    for r, n in enumerate(lens):
        k, v = np.zeros((layers, n, H, d)), np.zeros((layers, n, H, d))
        for li in range(layers):
            for h in range(H):
                if r < len(SHORT):
                    q[li, r, h * G:(h + 1) * G], k[li, :, h], v[li, :, h] = grid_case(rng, n, d, G)
                elif n and li == h == 0:  # rows of one head for all: only the lengths matter here
                    k[:, :], v[:, :] = (grid_rows(rng, n, d, low, 0.25)[None, :, None] for low in (0, -8))
        if n:
            ctx.append([r], dev(k[None]), dev(v[None]))
        given.append((k, v))
    if accumulate:
        ctx.track_weights()
    out, lse = ctx.decode_attention(dev(q), scale=GRID_SCALE, accumulate=accumulate)
    ctx.sync()
    out, lse = np64(out), np64(lse)
    worst = np.zeros(3)
    for li in range(layers):
        w = np64(dense_weights(ctx, li, 16)) if accumulate else None
        for r, n in enumerate(SHORT):
            for h in range(H):
                hs = slice(h * G, (h + 1) * G)
                args = q[li, r, hs], given[r][0][li, :, h], given[r][1][li, :, h]
                o, ll, a = step(*args, GRID_SCALE)
                bo, bl, ba = int4_grid_bounds(*args)
                errs = [np.abs(out[li, r, hs] - o) / (bo + 1e-300), np.abs(lse[li, r, hs] - ll) / bl]
                if accumulate:
                    errs.append(np.abs(w[r, h, :n] - a.sum(0)) / (ba.sum(0) + (G + 1) * U * a.sum(0)))
                worst[:len(errs)] = np.maximum(worst[:len(errs)], [e.max() for e in errs])
                assert all((e <= 1).all() for e in errs), (li, r, h, [float(e.max()) for e in errs])
    print(worst)
    ctx.close()


@pytest.mark.parametrize("accumulate", [False, True], ids=["step", "weights"])
@pytest.mark.parametrize("lens,layers,H,G", [([1, 31, 4097], 1, 2, 4), ([32768], 1, 8, 4), ([32767, 20000], 1, 4, 8),
                                             ([9001, 0, 17, 8999, 7000, 5000, 9000, 4999], 1, 8, 8),
                                             ([70, 333, 64, 5] * 16, 7, 8, 2), ([2049, 1000, 33] * 12, 1, 8, 1)], ids=str)
def test_a_zero_query_is_the_mean_of_every_row(lens, layers, H, G, accumulate):
    d = 128
    ctx = make(lens, layers=layers, H=H, G=G, d=d)
    rng = np.random.default_rng(sum(lens))
    pool = grid_rows(rng, max(lens), d, 0, 1.0)  # whole numbers from 0 to 15
    for r, n in enumerate(lens):
        if n:
            v = dev(np.roll(pool, r, 0)[:n])[None, None, :, None].expand(1, layers, n, H, d).contiguous()
            ctx.append([r], v, v)
    if accumulate:
        ctx.track_weights()
    out, lse = ctx.decode_attention(torch.zeros((layers, len(lens), H * G, d), dtype=torch.bfloat16, device="cuda"),
                                    accumulate=accumulate)
    ctx.sync()
    out, lse = np64(out), np64(lse)
    w = np64(dense_weights(ctx, layers - 1, max(lens))) if accumulate else None
    for r, n in enumerate(lens):
        if not n:
            assert not out[:, r].any() and np.isneginf(lse[:, r]).all()
            continue
        mean = np.roll(pool, r, 0)[:n].mean(0)
        assert (np.abs(out[:, r] - mean) <= 6 * U * mean).all(), (r, n)
        assert (np.abs(lse[:, r] - np.log(n)) <= 4 * U * (1 + np.log(n))).all(), (r, n)
        if accumulate:  # exp2 of -log2 n: its 4 u, and the roundings of log2 and lse
            assert (np.abs(w[r, :, :n] - G / n) <= (6 + 2 * np.log2(n) + G) * U * G / n).all(), (r, n)
    ctx.close()
