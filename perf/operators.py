"""Cases and plain forms of the 4-bit cache, of decode attention over it, of decode attention that accumulates the
attention weights, and of the eviction round that selects by them.

Every case is one call (or the few calls that belong together) of a serving loop:

* ``cache4``: a chunk of prompt rows is appended to a 4-bit cache, read back densely and the requests are released;
* ``attend``: one decode step of grouped-query attention over the cached rows (``cache``: int4, bf16 or f32), with
  ``accumulate`` also adding each row's attention weight to the cache's weights;
* ``evict``: the next window of rows is appended, the weights of the step arrive and one round keeps the best rows.

The 4-bit form of a row of d values: four groups of d/4 channels; lo = min and hi = max of a group,
s = (hi - lo)/15 rounded up to four significant bits, code = rint((x - lo)/s), value = lo + s*code.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 16
HOT, HOT_SCALE = 4, 8.0  # outlier channels of keys and values


def _lens(case):
    """Cached rows of each request (attend) or rows kept (evict), the same for every seed."""
    r, lo, hi = case["requests"], case["rows_min"], case["rows_max"]
    if lo == hi:
        return [hi] * r
    g = random.Random(1004 + r)
    out = [g.randint(lo, hi) for _ in range(r)]
    out[g.randrange(r)] = hi
    return out


def listed():
    return [
        # a prompt chunk of a busy server: 32 requests of 1024 tokens
        {"name": "cache4 prompt chunk", "op": "cache4", "requests": 32, "layers": 4, "kv_heads": 8, "dim": 128, "tokens": 1024},
        # the last tokens of short prompts, a length off the page, small heads: latency counts
        {"name": "cache4 short odd", "op": "cache4", "requests": 5, "layers": 2, "kv_heads": 2, "dim": 64, "tokens": 37},
        # the decode step of a serving batch after a round: 128 requests at 2048 rows, 32 query heads
        {"name": "attend int4 serving", "op": "attend", "cache": "int4", "accumulate": False, "requests": 128, "layers": 4,
         "kv_heads": 8, "group": 4, "dim": 128, "rows_min": 2048, "rows_max": 2048},
        # one request at the longest length, one layer per call as a model makes it
        {"name": "attend int4 one long", "op": "attend", "cache": "int4", "accumulate": False, "requests": 1, "layers": 1,
         "kv_heads": 8, "group": 4, "dim": 128, "rows_min": 32768, "rows_max": 32768},
        # requests of every age, 8 query heads on a KV head
        {"name": "attend int4 ragged acc", "op": "attend", "cache": "int4", "accumulate": True, "requests": 64, "layers": 1,
         "kv_heads": 8, "group": 8, "dim": 128, "rows_min": 4096, "rows_max": 32768},
        # the smallest decode step, an odd length: latency
        {"name": "attend int4 tiny acc", "op": "attend", "cache": "int4", "accumulate": True, "requests": 1, "layers": 1,
         "kv_heads": 2, "group": 1, "dim": 64, "rows_min": 253, "rows_max": 253},
        # the serving batch on the bf16 cache, its weights kept for the next round
        {"name": "attend bf16 serving acc", "op": "attend", "cache": "bf16", "accumulate": True, "requests": 128, "layers": 2,
         "kv_heads": 8, "group": 4, "dim": 128, "rows_min": 2048, "rows_max": 2048},
        # a few requests of very different lengths, one layer per call
        {"name": "attend bf16 few acc", "op": "attend", "cache": "bf16", "accumulate": True, "requests": 4, "layers": 1,
         "kv_heads": 8, "group": 4, "dim": 128, "rows_min": 700, "rows_max": 8191},
        # fp32 cache, multi-head
        {"name": "attend f32 acc", "op": "attend", "cache": "f32", "accumulate": True, "requests": 16, "layers": 2,
         "kv_heads": 4, "group": 2, "dim": 64, "rows_min": 100, "rows_max": 1500},
        # the serving round: 2048 + 64 rows back to 2048, the newest 64 always kept
        {"name": "evict serving", "op": "evict", "requests": 128, "layers": 4, "kv_heads": 8, "dim": 128, "prompt": 1024,
         "rows_min": 2048, "rows_max": 2048, "window": 64, "recent": 64, "hole_fill": False},
        # ragged requests that each bring a long window
        {"name": "evict ragged long", "op": "evict", "requests": 16, "layers": 2, "kv_heads": 8, "dim": 128, "prompt": 300,
         "rows_min": 2000, "rows_max": 9000, "window": 6144, "recent": 256, "hole_fill": False},
        # hole filling on a small odd cache: latency
        {"name": "evict small holes", "op": "evict", "requests": 3, "layers": 2, "kv_heads": 2, "dim": 64, "prompt": 16,
         "rows_min": 61, "rows_max": 333, "window": 48, "recent": 8, "hole_fill": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["cache4", "attend", "attend", "attend", "evict", "evict"])
    dim = rng.choice([64, 128, 128])
    if op == "cache4":
        case = {"op": op, "requests": _log(rng, 1, 48), "layers": rng.randint(1, 4), "kv_heads": rng.choice([1, 2, 4, 8]),
                "dim": dim, "tokens": _log(rng, 1, 1500)}
        while case["requests"] * case["layers"] * case["kv_heads"] * case["tokens"] > 1_000_000:
            case["tokens"] = max(1, case["tokens"] // 2)
        return case
    if op == "attend":
        cache = rng.choice(["int4", "int4", "bf16", "f32"])
        hi = _log(rng, 1, 32768)
        case = {"op": op, "cache": cache, "accumulate": rng.random() < 0.6, "requests": _log(rng, 1, 128), "layers": rng.randint(1, 3),
                "kv_heads": rng.choice([1, 2, 3, 8]), "group": rng.choice([1, 2, 4, 8]), "dim": dim,
                "rows_min": rng.choice([0, hi // 3, hi]), "rows_max": hi}
        if cache != "int4":
            case["accumulate"] = True
        while case["requests"] * case["layers"] * case["kv_heads"] * hi > 8_000_000 and case["requests"] > 1:
            case["requests"] //= 2
        return case
    lo = rng.randint(20, 400)
    case = {"op": op, "requests": _log(rng, 1, 64), "layers": rng.randint(1, 4), "kv_heads": rng.choice([1, 2, 5, 8]), "dim": dim,
            "prompt": rng.randint(0, 16), "rows_min": lo, "rows_max": lo + _log(rng, 1, 8000), "window": 16 * _log(rng, 1, 300),
            "recent": rng.choice([0, 1, 16, 100]), "hole_fill": rng.random() < 0.4}
    while case["requests"] * case["layers"] * case["kv_heads"] * (case["rows_max"] + case["window"]) > 8_000_000 and case["requests"] > 1:
        case["requests"] //= 2
    return case


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(1000 + 7 * int(seed))


def _hot(case, seed):
    """Channel scale [layers, 1, kv_heads, dim] with a few outlier channels per head."""
    g = torch.Generator().manual_seed(77 + int(seed))
    u = torch.rand((case["layers"], 1, case["kv_heads"], case["dim"]), generator=g)
    top = u.topk(HOT, dim=-1).indices
    return torch.ones_like(u).scatter_(-1, top, HOT_SCALE).cuda()


def _rows(case, gen, hot, n, dtype):
    """n rows of keys (or values) of every layer and KV head: [layers, n, kv_heads, dim]."""
    x = torch.randn((case["layers"], n, case["kv_heads"], case["dim"]), generator=gen, device="cuda")
    return (x * hot).to(dtype)


def _type(case):
    return torch.float32 if case.get("cache") == "f32" else torch.bfloat16


def _requests(case, seed, lens):
    """(k, v) rows of each request in turn, then the generator that drew them."""
    gen, hk, hv = _gen(seed), _hot(case, seed), _hot(case, seed + 5000)
    for n in lens:
        yield _rows(case, gen, hk, n, _type(case)), _rows(case, gen, hv, n, _type(case)), gen


def _queries(case, seed):
    g = torch.Generator(device="cuda").manual_seed(9_000_001 + int(seed))
    shape = (case["layers"], case["requests"], case["kv_heads"] * case["group"], case["dim"])
    return torch.randn(shape, generator=g, device="cuda").to(_type(case))


def _pages(rows):
    return (rows + PAGE - 1) // PAGE


# -------------------------------------------------------- the 4-bit row, 32 bits --

def _code4(x):
    """Codes (uint8, two to a byte, the lower channel in the low bits), steps and lows of rows x [..., dim]."""
    g = x.float().unflatten(-1, (4, -1))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    fifteen = torch.full_like(lo, 15.0)  # a tensor: a division by a number is a product with its rounded inverse
    r = (hi - lo) / fifteen
    s = ((r.view(torch.int32) + 0xFFFFF) & ~0xFFFFF).view(torch.float32)  # up to 4 significant bits
    s = torch.where(r >= 2.0 ** -100, s, torch.zeros_like(s))
    c = torch.where(s > 0, torch.round((g - lo) / torch.where(s > 0, s, torch.ones_like(s))), torch.zeros_like(g))
    c = c.to(torch.uint8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), s.squeeze(-1).bfloat16(), lo.squeeze(-1).bfloat16()


def _value4(code, s, lo):
    c = torch.stack((code & 15, code >> 4), -1).flatten(-2).float().unflatten(-1, (4, -1))
    return (lo.float().unsqueeze(-1) + s.float().unsqueeze(-1) * c).flatten(-2)


# ---------------------------------------------------------------- prepare --

def prepare(case, seed):
    return {"cache4": _prepare_cache4, "attend": _prepare_attend, "evict": _prepare_evict}[case["op"]](case, seed)


def _context(case, pages, longest, dtype):
    from decode_kv_cache_paged_b200 import Context, ContextSpec
    spec = ContextSpec(num_requests=case["requests"], num_layers=case["layers"], num_kv_heads=case["kv_heads"],
                       head_dim=case["dim"], max_seq_len=max(PAGE, PAGE * _pages(longest)), num_pages=max(1, pages),
                       num_q_heads=case["kv_heads"] * case.get("group", 1))
    return Context(spec, dtype=dtype)


def _prepare_cache4(case, seed):
    n, r = case["tokens"], case["requests"]
    k = torch.empty((r, case["layers"], n, case["kv_heads"], case["dim"]), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    for i, (kr, vr, _) in enumerate(_requests(case, seed, [n] * r)):
        k[i], v[i] = kr, vr
    state = {"case": case, "k": k, "v": v, "ids": np.arange(r, dtype=np.int32), "none": np.zeros(r, np.int32), "next": 0}
    if own:
        state["ctx"] = _context(case, r * _pages(n), n, "int4")
    return state


def _prepare_attend(case, seed):
    lens = _lens(case)
    longest, r, ly, h, d = max(lens), case["requests"], case["layers"], case["kv_heads"], case["dim"]
    pages = sum(_pages(n) for n in lens)
    state = {"case": case, "q": _queries(case, seed), "decay": 0.875}
    w0 = torch.rand((ly, max(1, pages), h, PAGE), generator=_gen(seed + 31), device="cuda") if case["accumulate"] else None
    if own:
        ctx = _context(case, pages, longest, {"int4": "int4", "bf16": torch.bfloat16, "f32": torch.float32}[case["cache"]])
        state["ctx"] = ctx
        for i, (k, v, _) in enumerate(_requests(case, seed, lens)):
            if lens[i]:
                ctx.append([i], k.unsqueeze(0), v.unsqueeze(0))
        if case["accumulate"]:
            ctx.track_weights().copy_(w0)
        return state
    # the plain form keeps the requests' rows dense: [layers, requests, kv_heads, longest, ...]
    if case["cache"] == "int4":
        for x in "kv":
            state[x] = (torch.zeros((ly, r, h, longest, d // 2), dtype=torch.uint8, device="cuda"),
                        torch.zeros((ly, r, h, longest, 4), dtype=torch.bfloat16, device="cuda"),
                        torch.zeros((ly, r, h, longest, 4), dtype=torch.bfloat16, device="cuda"))
    else:
        for x in "kv":
            state[x] = torch.zeros((ly, r, h, longest, d), dtype=_type(case), device="cuda")
    for i, rows in enumerate(_requests(case, seed, lens)):
        for x, y in zip("kv", rows):
            y = y.transpose(1, 2)  # [layers, kv_heads, n, dim]
            if case["cache"] == "int4":
                for whole, part in zip(state[x], _code4(y)):
                    whole[:, i, :, :lens[i]] = part
            else:
                state[x][:, i, :, :lens[i]] = y
    state["lens"] = torch.tensor(lens, device="cuda")
    if case["accumulate"]:
        state["w"] = w0
        at, base = [], 0  # page and place of every cached row, in the order of requests and rows
        for n in lens:
            at.append(torch.arange(n) + base * PAGE)
            base += _pages(n)
        state["at"] = torch.cat(at).cuda()
    return state


def _evict_sizes(case):
    keep = [max(n, case["prompt"] + 1) for n in _lens(case)]
    return keep, max(keep) + case["window"], sum(_pages(n) for n in keep), case["window"] // PAGE


def _prepare_evict(case, seed):
    keep, longest, filled, extra = _evict_sizes(case)
    r, ly, h, d, e, p = case["requests"], case["layers"], case["kv_heads"], case["dim"], case["window"], case["prompt"]
    pages = filled + r * extra
    bf16 = torch.bfloat16
    kw = torch.empty((r, ly, e, h, d), dtype=bf16, device="cuda")
    vw = torch.empty_like(kw)
    # weights as attention leaves them: spread over some orders of magnitude, a few rows with the same weight
    w_in = torch.exp(2.0 * torch.randn((ly, pages, h, PAGE), generator=_gen(seed + 31), device="cuda")).mul_(64).round_().div_(64)
    state = {"case": case, "kw": kw, "vw": vw, "w_in": w_in, "ids": np.arange(r, dtype=np.int32), "keep": np.array(keep, np.int32)}
    rows = _requests(case, seed, keep)
    if own:
        import decode_kv_cache_paged_b200 as kvc
        ctx = _context(case, pages, longest, bf16)
        ctx.k_pool.zero_()
        ctx.v_pool.zero_()
        ctx.set_option(kvc.KVC_OPT_RECENT_TOKENS, case["recent"])
        state["ctx"], state["w"] = ctx, ctx.track_weights()
        for i, (k, v, gen) in enumerate(rows):
            if p:
                ctx.append([i], k[:, :p].contiguous().unsqueeze(0), v[:, :p].contiguous().unsqueeze(0), protect=True)
            if keep[i] > p:
                ctx.append([i], k[:, p:].contiguous().unsqueeze(0), v[:, p:].contiguous().unsqueeze(0))
    else:
        state["kp"] = torch.zeros((ly, pages, h, PAGE, d), dtype=bf16, device="cuda")
        state["vp"] = torch.zeros_like(state["kp"])
        state["pos"] = torch.full((ly, pages, h, PAGE), -1, dtype=torch.int32, device="cuda")
        state["w"] = torch.zeros((ly, pages, h, PAGE), device="cuda")
        table = torch.zeros((r, _pages(longest)), dtype=torch.int64)
        base, tail = 0, filled
        for i, (k, v, gen) in enumerate(rows):
            n = keep[i]
            # the protected rows and the others arrive in two calls: the pages are the same
            table[i, :_pages(n)] = torch.arange(base, base + _pages(n))
            table[i, _pages(n):_pages(n) + extra] = torch.arange(tail, tail + extra)
            s = torch.arange(n, device="cuda")
            pg, off = base + s // PAGE, s % PAGE
            state["kp"][:, pg, :, off] = k.transpose(0, 1)
            state["vp"][:, pg, :, off] = v.transpose(0, 1)
            state["pos"][:, pg, :, off] = s.int().view(-1, 1, 1)
            base, tail = base + _pages(n), tail + extra
        state["table"] = table.cuda()
        state["n"] = torch.tensor(keep, device="cuda")
        state["next"] = torch.tensor(keep, device="cuda")
    for i in range(r):
        kw[i] = torch.randn(kw[i].shape, generator=gen, device="cuda").to(bf16)
        vw[i] = torch.randn(vw[i].shape, generator=gen, device="cuda").to(bf16)
    return state


# -------------------------------------------------------------------- run --

def run(state):
    return {"cache4": _run_cache4, "attend": _run_attend, "evict": _run_evict}[state["case"]["op"]](state)


def _run_cache4(state):
    case = state["case"]
    if own:
        ctx = state["ctx"]
        ctx.append(state["ids"], state["k"], state["v"])
        out = [ctx.gather_dense(layer, cap=case["tokens"]) for layer in range(case["layers"])]
        ctx.compress("random", state["none"], 0)  # releases the requests
        return {"k": [o[0] for o in out], "v": [o[1] for o in out], "pos": [o[2] for o in out]}
    k, v = (_value4(*_code4(state[x])).permute(1, 0, 3, 2, 4) for x in "kv")  # [layers, requests, kv_heads, tokens, dim]
    n, r, h = case["tokens"], case["requests"], case["kv_heads"]
    pos = (torch.arange(n, dtype=torch.int32, device="cuda") + state["next"]).expand(r, h, n).contiguous()
    state["next"] += n
    return {"k": list(k.contiguous()), "v": list(v.contiguous()), "pos": [pos] * case["layers"]}


def _run_attend(state):
    case = state["case"]
    if own:
        ctx = state["ctx"]
        if not case["accumulate"]:
            return ctx.decode_attention(state["q"])
        out, lse = ctx.decode_attention(state["q"], accumulate=True, decay=state["decay"])
        return out, lse, ctx.weights
    ly, r, h, g, d = case["layers"], case["requests"], case["kv_heads"], case["group"], case["dim"]
    k, v = (_value4(*state[x]) if case["cache"] == "int4" else state[x].float() for x in "kv")
    longest = k.shape[3]
    gone = torch.arange(longest, device="cuda") >= state["lens"].view(r, 1, 1, 1)
    if longest == 0:
        out = torch.zeros((ly, r, h * g, d), device="cuda")
        lse = torch.full((ly, r, h * g), -math.inf, device="cuda")
        return (out, lse, state["w"]) if case["accumulate"] else (out, lse)
    s = torch.matmul(state["q"].float().view(ly, r, h, g, d), k.transpose(-1, -2)) / math.sqrt(d)
    s.masked_fill_(gone, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    out = torch.matmul(p, v).view(ly, r, h * g, d)
    lse = (torch.log(total) + top).view(ly, r, h * g)
    if not case["accumulate"]:
        return out, lse
    new = p.sum(3).permute(0, 2, 1, 3)[:, :, ~gone.view(r, longest)]  # [layers, kv_heads, rows]
    w = state["w"].permute(0, 2, 1, 3).reshape(ly, h, -1)
    w[:, :, state["at"]] = w[:, :, state["at"]] * state["decay"] + new
    state["w"] = w.view(ly, h, -1, PAGE).permute(0, 2, 1, 3).contiguous()
    return out, lse, state["w"]


def _run_evict(state):
    case = state["case"]
    if own:
        ctx = state["ctx"]
        ctx.append(state["ids"], state["kw"], state["vw"])
        state["w"].copy_(state["w_in"])  # the attention of the step has written its weights
        ctx.compress("attention", state["keep"], 0, compaction="hole_fill" if case["hole_fill"] else "ordered")
        return ctx.k_pool, ctx.v_pool, ctx.state_tensors()["pos_map"], state["w"]
    ly, h, e, p = case["layers"], case["kv_heads"], case["window"], case["prompt"]
    table, n, r = state["table"], state["n"], case["requests"]
    kp, vp, pos, w = state["kp"], state["vp"], state["pos"], state["w"]
    # the window's rows
    t = torch.arange(e, device="cuda")
    slot = n.view(r, 1) + t
    pg, off = table.gather(1, slot // PAGE), slot % PAGE
    kp[:, pg, :, off] = state["kw"].permute(0, 2, 1, 3, 4)
    vp[:, pg, :, off] = state["vw"].permute(0, 2, 1, 3, 4)
    pos[:, pg, :, off] = (state["next"].view(r, 1) + t).int().view(r, e, 1, 1)
    state["next"] = state["next"] + e
    w.copy_(state["w_in"])
    # every slot of every segment [requests, layers, kv_heads, slots]: its row in the pools
    most = int(case["rows_max"] if case["rows_max"] > p else p + 1) + e
    slot = torch.arange(most, device="cuda")
    row = (table[:, slot // PAGE].view(r, 1, 1, most) + torch.arange(ly, device="cuda").view(1, ly, 1, 1) * kp.shape[1]) * h
    row = (row + torch.arange(h, device="cuda").view(1, 1, h, 1)) * PAGE + slot % PAGE
    end, budget = (n + e).view(r, 1, 1, 1), (n - p).view(r, 1, 1, 1)
    cand = ((slot >= p) & (slot < end)).expand(row.shape)
    at = pos.view(-1)[row]
    score = w.view(-1)[row]
    newest = at >= state["next"].view(r, 1, 1, 1) - budget.clamp(max=case["recent"])
    score = torch.where(newest, math.inf, score)
    score = torch.where(cand, score, -math.inf)
    by_pos = at.sort(dim=-1, stable=True).indices
    order = by_pos.gather(-1, score.gather(-1, by_pos).sort(dim=-1, descending=True, stable=True).indices)
    kept = torch.zeros(row.shape, dtype=torch.bool, device="cuda")
    kept.scatter_(-1, order, (slot < budget).expand(row.shape).contiguous())
    if case["hole_fill"]:
        below = slot < p + budget
        src, dst = row[kept & ~below], row[cand & ~kept & below]
    else:
        rank = kept.cumsum(-1) - 1 + p
        src = row[kept]
        dst = row.gather(-1, rank.clamp(min=0))[kept]
    for x in (kp.view(-1, case["dim"]), vp.view(-1, case["dim"]), pos.view(-1), w.view(-1)):
        x[dst] = x[src]
    # the pages past the kept rows are free; the next window takes the last ones freed first
    extra = e // PAGE
    cols = ((n + PAGE - 1) // PAGE).view(r, 1) + torch.arange(extra, device="cuda")
    table.scatter_(1, cols, table.gather(1, cols).flatten().flip(0).view(r, extra))
    return kp, vp, pos, w


# ------------------------------------------------------------------- work --

def work(case):
    r, ly, h, d = case["requests"], case["layers"], case["kv_heads"], case["dim"]
    row4 = d // 2 + 16
    if case["op"] == "cache4":
        rows = r * ly * h * case["tokens"]
        # read K and V, write the 4-bit rows, read them, write 32-bit rows; a position written and read
        return {"bytes": rows * (2 * (2 * d + 2 * row4 + 4 * d) + 12), "flops": rows * 2 * 6 * d}
    if case["op"] == "attend":
        rows = sum(_lens(case)) * ly * h
        per = 2 * {"int4": row4, "bf16": 2 * d, "f32": 4 * d}[case["cache"]] + (8 if case["accumulate"] else 0)
        heads = r * ly * h * case["group"]
        return {"bytes": rows * per + heads * (d * (8 if case["cache"] == "f32" else 6) + 4),
                "flops": rows * case["group"] * (4 * d + 8)}
    keep = _evict_sizes(case)[0]
    segs, e, p = ly * h, case["window"], case["prompt"]
    moved = [n - p for n in keep]
    if case["hole_fill"]:  # a hole for each row kept past the new length, about
        moved = [(n - p) * e / (n - p + e) for n in keep]
    rows = segs * sum(moved)
    new = segs * r * e
    cand = segs * sum(n - p + e for n in keep)
    return {"bytes": new * (8 * d + 4) + cand * 4 + rows * (8 * d + 16) + segs * 8 * sum(n + e for n in keep), "flops": cand}


# ------------------------------------------------------------------ exact --

def _exact4(x):
    """Values of 4-bit rows, from the definition, in 64 bits."""
    shape = x.shape
    x = x.double().reshape(*shape[:-1], 4, shape[-1] // 4)
    lo = x.min(-1, keepdim=True).values
    step = (x.max(-1, keepdim=True).values - lo).div(torch.tensor(15.0, dtype=torch.float64, device=x.device))
    m, ex = torch.frexp(step)
    up = torch.ldexp(torch.ceil(m * 16) / 16, ex)
    up = up * (step >= 2.0 ** -100)
    code = torch.round(torch.nan_to_num((x - lo) / up, nan=0.0, posinf=0.0, neginf=0.0))
    return (lo + up * code).reshape(shape)


def exact(case, seed):
    if case["op"] == "evict":
        return None  # rows and weights move as they are; nothing is computed
    if case["op"] == "cache4":
        k, v = [], []
        for kr, vr, _ in _requests(case, seed, [case["tokens"]] * case["requests"]):
            k.append(_exact4(kr).transpose(1, 2).float().cpu())  # a value has fewer than 24 bits
            v.append(_exact4(vr).transpose(1, 2).float().cpu())
        k, v = torch.stack(k, 1), torch.stack(v, 1)
        if case["tokens"] * case["requests"] * case["layers"] * case["kv_heads"] > 200_000:
            return {"k": list(k), "v": list(v), "pos": [None] * case["layers"]}
        return {"k": list(k.double()), "v": list(v.double()), "pos": [None] * case["layers"]}
    lens = _lens(case)
    r, ly, h, g, d = case["requests"], case["layers"], case["kv_heads"], case["group"], case["dim"]
    if sum(lens) * ly * h * g > 200_000_000:
        return None
    q = _queries(case, seed).double().reshape(ly, r, h, g, d)
    out = torch.zeros((ly, r, h, g, d), dtype=torch.float64, device="cuda")
    lse = torch.full((ly, r, h, g), -math.inf, dtype=torch.float64, device="cuda")
    pages = max(1, sum(_pages(n) for n in lens))
    w = torch.rand((ly, pages, h, PAGE), generator=_gen(seed + 31), device="cuda").double() if case["accumulate"] else None
    base = 0
    for i, (k, v, _) in enumerate(_requests(case, seed, lens)):
        n = lens[i]
        if n:
            k, v = (_exact4(x) if case["cache"] == "int4" else x.double() for x in (k, v))  # [layers, n, kv_heads, dim]
            s = torch.einsum("lhgd,lnhd->lhgn", q[:, i], k) * d ** -0.5
            lse[:, i] = torch.logsumexp(s, -1)
            a = torch.exp(s - lse[:, i].unsqueeze(-1))
            out[:, i] = torch.einsum("lhgn,lnhd->lhgd", a, v)
            if w is not None:
                part = w[:, base:base + _pages(n)].transpose(1, 2).reshape(ly, h, -1)
                part[:, :, :n] = 0.875 * part[:, :, :n] + a.sum(2)
                w[:, base:base + _pages(n)] = part.reshape(ly, h, -1, PAGE).transpose(1, 2)
        base += _pages(n)
    out, lse = out.reshape(ly, r, h * g, d), lse.reshape(ly, r, h * g)
    return (out, lse) if w is None else (out, lse, w)
