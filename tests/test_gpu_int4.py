"""The 4-bit cache: its rows bit for bit, decode attention over them, rounds that move them.

Tolerance of the attention (u = 2^-24).  The scores' products of codes and the integer parts of the query are exact, and
so are their sums (integers below 2^21); the rest of the query is at most 1/2 beside integers up to 2047 and its 16-term
products may lose 2u of their largest each (with 8 heads they are added to the integers' sums and may lose 2u of those).
s and lo join them in fp32: 12 roundings per score, scaling, the subtraction of the maximum and exp2 add four.  With A = max_j scale*(sum_i |q_i| step code_ji + sum_g |lo_jg| sum_{i in g} |q_i|):
  score error  ds <= 16 u A + 2u*|s - m| + 4u; 4 (d/16 + 5) u A is used, which is above it.
A weight enters the second product as three bf16 numbers that hold all of its bits; the tensor cores may truncate 2u of the
largest of 16 products each, in a chain of at most 6, and the running sums take L/32 additions, the merges 64 more:
  out error    <= 3 max_j|v_jc| * (2 ds + 2 * 2^-18 + 2*(L/16 + 64)*2u),  (2^-18 = 64u covers the products' truncation)
  lse error    <= ds + 2^-18 + (L/16 + 64)*2u + 4u|lse|."""
import numpy as np
import pytest
import torch

import rows4
from decode_kv_cache_paged_b200 import KVC_ERR_STATE, KVC_ERR_UNSUPPORTED, Context, ContextSpec, KvcError

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def make(lens, layers=1, H=2, G=1, d=128, dtype="int4", extra_pages=4, room=0, window=0, device="cuda"):
    longest = max(max(lens) + room, 16)
    spec = ContextSpec(num_requests=len(lens), num_layers=layers, num_kv_heads=H, head_dim=d,
                       max_seq_len=(longest + 15) // 16 * 16, num_q_heads=H * G, query_window=window,
                       num_pages=sum((n + room + 15) // 16 for n in lens) + extra_pages)
    return Context(spec, dtype=dtype, device=device)


def rows(n, layers, H, d, seed, kind="normal", dtype=torch.bfloat16):
    """K (or V) rows [1, layers, n, H, d]."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((1, layers, n, H, d), generator=g, device="cuda")
    if kind == "hot":
        x[..., 3::d // 4] *= 8
    elif kind == "ties":  # steps of 1 and values on halves: every other code is a tie
        x = torch.randint(0, 31, x.shape, generator=g, device="cuda") / 2
        x[..., 0::d // 4] = 0
        x[..., 1::d // 4] = 15
    elif kind == "offset":
        x = x * 0.25 + 100
    elif kind == "constant":
        x = x[..., :1].expand(x.shape).contiguous()
    elif kind == "zero":
        x = torch.zeros_like(x)
    elif kind == "wide":
        x = x * 2.0 ** torch.randint(-40, 40, x.shape[:-1] + (1,), generator=g, device="cuda")
    elif kind == "edge":  # ranges around the smallest step and the largest one
        e = torch.randint(0, 4, x.shape[:-1] + (1,), generator=g, device="cuda")
        x = torch.where(e == 0, x * 2.0 ** -54, torch.where(e == 1, x * 2.0 ** -70, torch.where(e == 2, x * 2.0 ** 58, x * 2.0 ** 90)))
    elif kind == "broken":
        bad = torch.randint(0, 200, x.shape, generator=g, device="cuda")
        x = torch.where(bad == 0, float("inf"), torch.where(bad == 1, float("-inf"), torch.where(bad == 2, float("nan"), x)))
    return x.to(dtype)


def fill(ctx, lens, seed=0, kind="hot", chunk=None):
    """Appends lens[i] rows to request i; returns the K and V rows given, per request [layers, n, H, d]."""
    s, out = ctx.spec, []
    for i, n in enumerate(lens):
        k = rows(n, s.num_layers, s.num_kv_heads, s.head_dim, seed + 10 * i, kind, ctx.dtype)
        v = rows(n, s.num_layers, s.num_kv_heads, s.head_dim, seed + 10 * i + 5, kind, ctx.dtype)
        step = chunk or max(n, 1)
        for t in range(0, n, step):
            ctx.append([i], k[:, :, t:t + step].contiguous(), v[:, :, t:t + step].contiguous())
        out.append((k[0], v[0]))
    return out


def np64(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["normal", "hot", "ties", "offset", "constant", "zero", "wide", "edge", "broken"])
def test_values_are_the_definitions(d, kind):
    """gather_dense returns exactly what the definition says, for every kind of row."""
    lens = [37, 1, 0, 64]
    ctx = make(lens, layers=2, H=3, d=d)
    given = fill(ctx, lens, seed=3, kind=kind, chunk=13)
    for layer in range(2):
        k, v, pos = ctx.gather_dense(layer)
        assert k.dtype == torch.float32
        for i, n in enumerate(lens):
            for got, x in ((k, given[i][0]), (v, given[i][1])):
                want = rows4.row_values(np64(x[layer]).transpose(1, 0, 2))
                have = got[i, :, :n].cpu().numpy()
                assert np.array_equal(np.isnan(have), np.isnan(want))
                assert np.array_equal(have[~np.isnan(want)], want[~np.isnan(want)].astype(np.float32))
                assert not got[i, :, n:].any()
            assert np.array_equal(pos[i, :, :n].cpu().numpy(), np.tile(np.arange(n), (3, 1)))
            assert (pos[i, :, n:] == -1).all()
    ctx.close()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["hot", "ties", "offset", "wide", "zero"])
def test_row_bytes_are_the_documented_ones(d, kind):
    ctx = make([20], H=2, d=d)
    (k, v), = fill(ctx, [20], seed=8, kind=kind)
    assert ctx.view().row_bytes == d // 2 + 16 == ctx.k_pool.shape[-1]
    bt = ctx.state_tensors()["block_table"].cpu()
    for pool, x, is_v in ((ctx.k_pool, k, False), (ctx.v_pool, v, True)):
        step, lo, codes = rows4.code_rows(np64(x[0]).transpose(1, 0, 2))
        z, mid = rows4.centres(step, lo) if is_v else (np.zeros_like(lo), lo)
        for j in (0, 15, 16, 19):
            raw = pool[0, int(bt[0, j // 16]), :, j % 16].cpu().numpy()  # [H, row bytes]
            head = raw[:, :16].copy().view(np.uint32)
            assert np.array_equal((head & 0xFFF00000).view(np.float32), step[:, j].astype(np.float32))
            assert np.array_equal(head >> 16 & 15, z[:, j].astype(np.uint32))
            have = (head << 16).view(np.float32).astype(np.float64)
            assert np.array_equal(have, mid[:, j])  # exactly: mid needs no rounding
            c = codes[:, j].reshape(2, d).astype(np.uint8)
            c = c if is_v else rows4.k_order(c)
            assert np.array_equal(raw[:, 16:], c[:, 0::2] | (c[:, 1::2] << 4))
    ctx.close()


def test_host_rows_and_ring_queries():
    """Rows from page-locked host memory; the query ring keeps bf16 queries."""
    ctx = make([40], H=2, G=4, d=64, window=8)
    k, v = (rows(40, 1, 2, 64, s).cpu().pin_memory() for s in (1, 2))
    q = rows(40, 1, 8, 64, 3)
    ctx.append([0], k, v, q)
    got = ctx.gather_dense(0)[0][0].cpu().numpy()[:, :40]
    assert np.array_equal(got, rows4.row_values(np64(k[0, 0]).transpose(1, 0, 2)).astype(np.float32))
    ring = ctx.state_tensors()["query_ring"][0, 0]
    assert torch.equal(ring, q[0, 0, 32:])  # slot = step mod 8
    ctx.close()


def check_attention(ctx, q, out, lse, layers, scale, tag=""):
    s = ctx.spec
    lens, _ = ctx.lengths()
    d, G = s.head_dim, s.num_q_heads // s.num_kv_heads
    worst = 0.0
    for li, layer in enumerate(layers):
        k, v, _ = ctx.gather_dense(layer, cap=int(max(lens.max(), 1)))
        for r, L in enumerate(lens):
            if L == 0:
                assert not out[li, r].any() and torch.isneginf(lse[li, r]).all(), tag
                continue
            for h in range(s.num_kv_heads):
                qq = np64(q[li, r, h * G:(h + 1) * G])
                kk, vv = np64(k[r, h, :L]), np64(v[r, h, :L])
                o, ll, _ = rows4.attention(qq, kk, vv, scale)
                lo = np.repeat(kk.reshape(L, 4, -1).min(-1), d // 4, -1)  # at least the group's lo in size, with 15 steps
                A = scale * (np.abs(qq) @ (np.abs(kk - lo) + np.abs(lo)).T)
                ss = scale * (qq @ kk.T)
                ds = (2 * (d / 16 + 1) + 8) * 2 * U * A.max(-1) + 2 * U * (ss.max(-1) - ss.min(-1)) + 4 * U
                chain = (L / 16 + 64) * 2 * U
                tol = 3 * np.abs(vv).max(0) * (2 * ds + 2 * 2.0 ** -18 + 2 * chain)[:, None] + 1e-30
                err = np.abs(np64(out[li, r, h * G:(h + 1) * G]) - o)
                assert np.all(err <= tol), (tag, layer, r, h, float((err / tol).max()))
                le = np.abs(np64(lse[li, r, h * G:(h + 1) * G]) - ll)
                assert np.all(le <= ds + 2.0 ** -18 + chain + 4 * U * np.abs(ll)), (tag, layer, r, h, float(le.max()))
                worst = max(worst, float((err / tol).max()))
    return worst


LENS = [0, 1, 2, 15, 16, 17, 31, 64, 65, 253, 1027]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_attention(G, d):
    ctx = make(LENS, layers=2, H=2, G=G, d=d)
    fill(ctx, LENS, seed=20)
    q = rows(len(LENS), 2, 2 * G, d, 5)[0]  # [layers, R, Hq, d]
    out, lse = ctx.decode_attention(q)
    ctx.sync()
    print(check_attention(ctx, q, out, lse, range(2), d ** -0.5))
    ctx.close()


@pytest.mark.parametrize("lens", [[4133], [9001, 40], [32768]], ids=str)
def test_attention_long(lens):
    ctx = make(lens, H=2, G=4)
    fill(ctx, lens, seed=30)
    q = rows(len(lens), 1, 8, 128, 6)[0]
    out, lse = ctx.decode_attention(q)
    ctx.sync()
    print(check_attention(ctx, q, out, lse, [0], 128 ** -0.5))
    ctx.close()


def test_attention_many_units():
    """More (layer, request, KV head) units than CTAs fit at a time; a subset of the layers; a scale."""
    lens = [100 + 13 * i for i in range(40)]
    ctx = make(lens, layers=4, H=8, G=4, d=64)
    fill(ctx, lens, seed=40)
    q = rows(len(lens), 2, 32, 64, 7)[0]
    out, lse = ctx.decode_attention(q, layer_begin=1, scale=0.3)
    ctx.sync()
    print(check_attention(ctx, q, out, lse, [1, 2], 0.3))
    ctx.close()


@pytest.mark.parametrize("G", [1, 4, 8])
def test_attention_one_warp_units(G):
    """Units enough for the form with one warp a unit: lengths around the pairs of pages a warp takes."""
    lens = [(7 * i) % 70 for i in range(60)]
    ctx = make(lens, layers=8, H=8, G=G, d=64)
    fill(ctx, lens, seed=45)
    q = rows(len(lens), 8, 8 * G, 64, 8)[0]
    out, lse = ctx.decode_attention(q)
    ctx.sync()
    print(check_attention(ctx, q, out, lse, range(8), 64 ** -0.5))
    ctx.close()


def test_unaligned_queries():
    """Queries on a 2-byte boundary, as the call allows, give the same bits."""
    ctx = make([70, 300], H=2, G=4)
    fill(ctx, [70, 300], seed=46)
    q = rows(2, 1, 8, 128, 9)[0].contiguous()
    a = ctx.decode_attention(q)
    odd = torch.empty(q.numel() + 1, dtype=q.dtype, device="cuda")[1:].view(q.shape)
    odd.copy_(q)
    assert odd.data_ptr() % 16 == 2
    b = ctx.decode_attention(odd)
    ctx.sync()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ctx.close()


def test_query_ranges():
    """Query values 30 binades apart, tiny and huge queries, and a zero query in one batch."""
    lens = [40, 90, 33, 50]
    ctx = make(lens, H=2, G=4)
    fill(ctx, lens, seed=47, kind="normal")
    q = rows(4, 1, 8, 128, 10)[0].float()
    q[:, 0] *= torch.where(torch.arange(128, device="cuda") % 3 == 0, 2.0 ** -30, 1.0)
    q[:, 1] *= 2.0 ** -100
    q[:, 2] *= 16.0
    q[:, 3] = 0
    q = q.bfloat16()
    out, lse = ctx.decode_attention(q)
    ctx.sync()
    print(check_attention(ctx, q, out, lse, [0], 128 ** -0.5))
    ctx.close()


def test_broken_queries_stay_in_their_rows():
    """An infinite or NaN query value makes its own head's row NaN and no other."""
    ctx = make([50], H=2, G=4)
    fill(ctx, [50], seed=48)
    q = rows(1, 1, 8, 128, 11)[0]
    want = ctx.decode_attention(q)
    for bad in (float("inf"), float("nan")):
        x = q.clone()
        x[0, 0, 5, 77] = bad
        out, lse = ctx.decode_attention(x)
        ctx.sync()
        keep = [i for i in range(8) if i != 5]
        assert torch.isnan(out[0, 0, 5]).all() and torch.isnan(lse[0, 0, 5])
        assert torch.equal(out[0, 0, keep], want[0][0, 0, keep]) and torch.equal(lse[0, 0, keep], want[1][0, 0, keep])
    ctx.close()


@pytest.mark.parametrize("kind", ["wide", "offset", "constant", "zero"])
def test_attention_value_ranges(kind):
    """Keys and values far from 1: the sums stay finite and within the bound."""
    lens = [70, 300]
    ctx = make(lens, H=2, G=4)
    s = ctx.spec
    for i, n in enumerate(lens):
        k = rows(n, 1, 2, 128, 50 + i, "hot" if kind == "wide" else kind)
        ctx.append([i], k, rows(n, 1, 2, 128, 60 + i, kind))
    q = rows(2, 1, 8, 128, 9)[0]
    out, lse = ctx.decode_attention(q)
    ctx.sync()
    print(check_attention(ctx, q, out, lse, [0], 128 ** -0.5))
    assert torch.isfinite(out).all()
    del s
    ctx.close()


def test_sharp_scores():
    """Scores hundreds apart: the running maximum moves by far more than a step, up and down."""
    lens = [600]
    ctx = make(lens, H=2, G=4)
    k = rows(600, 1, 2, 128, 70)
    k[:, :, 77] *= 20
    k[:, :, 399] *= 60
    ctx.append([0], k, rows(600, 1, 2, 128, 71))
    q = rows(1, 1, 8, 128, 10)[0] * 4
    out, lse = ctx.decode_attention(q)
    ctx.sync()
    print(check_attention(ctx, q, out, lse, [0], 128 ** -0.5))
    ctx.close()


def test_what_lies_past_the_rows_does_not_matter():
    """Garbage (NaN steps among it) behind the last row of a page, and in free pages, changes no bit."""
    lens = [5, 33, 250]
    q = rows(3, 1, 8, 128, 11)[0]
    got = []
    for junk in (0, 255):
        ctx = make(lens, H=2, G=4)
        ctx.k_pool.fill_(junk)
        ctx.v_pool.fill_(junk)
        fill(ctx, lens, seed=80)
        got.append(ctx.decode_attention(q))
        ctx.sync()
        ctx.close()
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert torch.isfinite(got[0][0]).all()


def test_a_broken_group_shows_only_where_it_is_read():
    """A NaN in one request's values leaves the other requests and KV heads as they were."""
    lens = [40, 40]
    ctx = make(lens, H=2, G=4)
    k, v = rows(40, 1, 2, 128, 90), rows(40, 1, 2, 128, 91)
    ctx.append([0], k, v)
    v2 = v.clone()
    v2[0, 0, 7, 1, 100] = float("nan")  # group 3 of KV head 1
    ctx.append([1], k, v2)
    q = rows(2, 1, 8, 128, 12)[0]
    q[:, 1] = q[:, 0]
    out, lse = ctx.decode_attention(q)
    ctx.sync()
    assert torch.equal(out[0, 0, :4], out[0, 1, :4]) and torch.equal(lse[0, 0], lse[0, 1])
    assert torch.isnan(out[0, 1, 4:, 96:]).all()
    assert torch.equal(out[0, 0, 4:, :96], out[0, 1, 4:, :96])
    ctx.close()


@pytest.mark.parametrize("G,layers,lens", [(8, 1, [9000, 0, 1, 16, 4097, 300, 8999, 5000]), (4, 2, [9001, 33, 0, 7000, 5000, 8000, 2, 9000]),
                                           (8, 3, [5000, 4999, 17, 0])])
def test_attention_more_ctas_than_fit(G, layers, lens):
    """Units split over more CTAs than fit the GPU at once, their partials merged by a second launch."""
    ctx = make(lens, layers=layers, H=8, G=G)
    fill(ctx, lens, seed=95)
    q = rows(len(lens), layers, 8 * G, 128, 19)[0]
    out, lse = ctx.decode_attention(q)
    ctx.sync()
    print(check_attention(ctx, q, out, lse, range(layers), 128 ** -0.5))
    ctx.close()


def test_split_steps_with_empty_and_broken_requests():
    """A few long requests (split over CTAs, merged by a second launch) beside an empty one, a short one and one with a
    broken key group: its heads are NaN, the others' outputs are the definition's."""
    lens = [20000, 0, 7, 4500]
    ctx = make(lens, H=2, G=4)
    fill(ctx, lens[:3], seed=92)
    k, v = rows(4500, 1, 2, 128, 93), rows(4500, 1, 2, 128, 94)
    k[0, 0, 4321, 1, 5] = float("nan")
    ctx.append([3], k, v)
    q = rows(4, 1, 8, 128, 18)[0]
    out, lse = ctx.decode_attention(q)
    ctx.sync()
    assert torch.isnan(out[0, 3, 4:]).all() and torch.isnan(lse[0, 3, 4:]).all()
    assert torch.isfinite(out[0, 3, :4]).all() and torch.isfinite(lse[0, 3, :4]).all()
    assert not out[0, 1].any() and torch.isneginf(lse[0, 1]).all()
    ctx2 = make(lens, H=2, G=4)
    fill(ctx2, lens[:3], seed=92)
    out2, lse2 = ctx2.decode_attention(q)
    ctx2.sync()
    assert torch.equal(out[0, :3], out2[0, :3]) and torch.equal(lse[0, :3], lse2[0, :3])
    check_attention(ctx2, q, out2, lse2, [0], 128 ** -0.5)
    ctx.close()
    ctx2.close()


@pytest.mark.parametrize("compaction", ["ordered", "hole_fill"])
@pytest.mark.parametrize("d", [64, 128])
def test_rounds_move_whole_rows(d, compaction):
    """After random rounds and appends every slot holds the values of the position that it names."""
    lens = [200, 77, 5200]
    ctx = make(lens, layers=2, H=2, d=d, room=32)
    given = fill(ctx, lens, seed=100)
    budgets = np.array([120, 64, 4096], np.int32)
    more = [[], [], []]
    for rnd in range(2):
        ctx.compress("random", budgets - 16 * rnd, 5 + rnd, compaction=compaction)
        k = rows(3 * 9, 2, 2, d, 200 + rnd).view(2, 3, 9, 2, d).transpose(0, 1).contiguous()
        ctx.append([0, 1, 2], k, k)
        for i in range(3):
            more[i].append(k[i])
    ctx.sync()
    now, _ = ctx.lengths()
    assert now.tolist() == [113, 57, 4089]
    for layer in range(2):
        gk, gv, gp = ctx.gather_dense(layer)
        for i in range(3):
            allk = np64(torch.cat([given[i][0]] + more[i], 1)[layer])  # [n, H, d] by position
            allv = np64(torch.cat([given[i][1]] + more[i], 1)[layer])
            for h in range(2):
                pos = gp[i, h, :now[i]].cpu().numpy()
                assert len(set(pos.tolist())) == now[i]
                assert np.array_equal(gk[i, h, :now[i]].cpu().numpy(), rows4.row_values(allk[pos, h]).astype(np.float32))
                assert np.array_equal(gv[i, h, :now[i]].cpu().numpy(), rows4.row_values(allv[pos, h]).astype(np.float32))
    q = rows(3, 2, 2, d, 13)[0]
    out, lse = ctx.decode_attention(q)
    ctx.sync()
    print(check_attention(ctx, q, out, lse, range(2), d ** -0.5))
    ctx.close()


def test_the_same_call_gives_the_same_bits():
    ctx = make([3000, 10], H=2, G=8)
    fill(ctx, [3000, 10], seed=110)
    q = rows(2, 1, 16, 128, 14)[0]
    a = ctx.decode_attention(q)
    b = ctx.decode_attention(q)
    ctx.sync()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ctx.close()


@pytest.mark.parametrize("dtype", ["int4", torch.bfloat16], ids=str)
def test_captured_step_follows_the_cache(dtype):
    """A captured step replays over the cache as it then stands: more rows, other queries."""
    lens = [100, 900]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ctx = make(lens, H=2, G=4, room=2000, dtype=dtype)
        fill(ctx, lens, seed=120)
        q = rows(2, 1, 8, 128, 15)[0]
        out, lse = ctx.decode_attention(q)  # the first call sets the kernels up
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            ctx.decode_attention(q, out=out, lse=lse)
        fill(ctx, [1500, 700], seed=130)
        q.copy_(rows(2, 1, 8, 128, 16)[0])
        graph.replay()
        side.synchronize()
        print(check_attention(ctx, q, out, lse, [0], 128 ** -0.5))
        side.synchronize()
    ctx.close()


@pytest.mark.parametrize("room", [0, 30000])
def test_two_captured_steps_share_the_context(room):
    """Two captured steps of other layers and queries, replayed one after the other in both orders."""
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ctx = make([700, 300], layers=2, H=2, G=4, room=room)
        fill(ctx, [700, 300], seed=125)
        qs = [rows(2, 1, 8, 128, 20 + i)[0] for i in range(2)]
        res = [ctx.decode_attention(qs[i], layer_begin=i) for i in range(2)]
        side.synchronize()
        graphs = []
        for i in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                ctx.decode_attention(qs[i], layer_begin=i, out=res[i][0], lse=res[i][1])
            graphs.append(g)
        for order in ((0, 1), (1, 0)):
            for o in res:
                o[0].zero_()
            for i in order:
                graphs[i].replay()
            side.synchronize()
            for i in range(2):
                check_attention(ctx, qs[i], res[i][0], res[i][1], [i], 128 ** -0.5)
        side.synchronize()
    ctx.close()


def test_pools_past_4_gb():
    """Row addresses past 2^32 bytes: the last layers of pools of 6 GB."""
    ctx = make([100, 47], layers=4, H=8, G=4, extra_pages=150000)
    assert ctx.k_pool.numel() > 6 * 10 ** 9
    given = fill(ctx, [100, 47], seed=135)
    w = ctx.track_weights()
    q = rows(2, 1, 32, 128, 30)[0]
    out, lse = ctx.decode_attention(q, layer_begin=3, accumulate=True)
    ctx.sync()
    print(check_attention(ctx, q, out, lse, [3], 128 ** -0.5))
    k, _, _ = ctx.gather_dense(3)
    assert np.array_equal(k[0, :, :100].cpu().numpy(), rows4.row_values(np64(given[0][0][3]).transpose(1, 0, 2)).astype(np.float32))
    assert abs(float(w[3].sum()) - 2 * 32) < 1e-2 and not w[:3].any()  # each query head's weights sum to 1
    ctx.compress("attention", np.array([40, 40], np.int32), 0)
    ctx.sync()
    assert ctx.lengths()[0].tolist() == [40, 40]
    ctx.close()


def test_refusals():
    ctx = make([20], H=2, G=3)
    q = rows(1, 1, 6, 128, 1)[0]
    with pytest.raises(KvcError) as e:
        ctx.decode_attention(q)
    assert e.value.status == KVC_ERR_UNSUPPORTED
    with pytest.raises(KvcError) as e:
        ctx.compress("beacon", np.array([4], np.int32), 0)
    assert e.value.status == KVC_ERR_STATE
    with pytest.raises(KvcError):
        ctx.update_beacons()
    with pytest.raises(ValueError):
        ctx.append([0], torch.zeros((1, 1, 2, 2, 128), device="cuda"), torch.zeros((1, 1, 2, 2, 128), device="cuda"))
    with pytest.raises(ValueError):
        ctx.decode_attention(q.float())
    ctx.close()
