"""The paged 4-bit memory's operators, as cases to measure: page tables, append and read-back, page
selection, and decode attention over requests of different lengths.

A page holds `page` tokens of one request (a memory block) for every kv head, in strips of 16 tokens.
A strip of one kv head is one run of bytes, with P = 64 or 128 dims a row and G = P / 32 groups:
    K codes   8 P bytes   the 32-bit word (token t, lane c < 4, group g) at word (4 t + c) G + g;
                          its nibble j is dim 32 g + 8 c + j
    V codes   8 P bytes   the 16-bit unit (token t = 8 p + 2 c + o, lane l < 8, group g) at unit
                          ((8 p + l) 4 + c) 2 G + 2 g + o;  its nibble j is dim 32 g + 4 l + j
    scales    64 G bytes  bf16 [token][K group 0 .. G-1, V group 0 .. G-1]
A code c + 8 stands for c s, c in -7 .. 7, s the group's scale.
"""
import math

import torch

own = False

STRIP = 16


# ---------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # one continuous-batching decode step: every running request gets one more token, a few idle
        {"name": "tables-decode-256", "op": "tables", "requests": 256, "longest": 32768, "page": 128, "tokens": 250},
        # prompts admitted together into a pool of small pages
        {"name": "tables-prompts-96k", "op": "tables", "requests": 33, "longest": 4096, "page": 24, "tokens": 98304},
        # one token of each of 64 requests written (InfLLM heads)
        {"name": "append-decode-64", "op": "append", "tokens": 64, "run": 1, "heads": 8, "dim": 128, "page": 128, "type": "bf16"},
        # a prompt chunk written, page summaries with it (InfLLM heads)
        {"name": "append-prompt-8k", "op": "append", "tokens": 8192, "run": 8192, "heads": 8, "dim": 128, "page": 128, "type": "bf16"},
        # ragged fp32 rows with MemLong's head size and Landmark's 50-token blocks
        {"name": "append-ragged-d100", "op": "append", "tokens": 777, "run": 111, "heads": 32, "dim": 100, "page": 50, "type": "f32"},
        # one long-context request (InfLLM 128K)
        {"name": "select-128k", "op": "select", "requests": 1, "longest": 131072, "heads": 8, "group": 4, "dim": 128, "page": 128, "k": 32, "sink": 128, "window": 4096, "type": "bf16"},
        # a batch of requests of every length (Landmark heads and blocks)
        {"name": "select-landmark-b16", "op": "select", "requests": 16, "longest": 32768, "heads": 32, "group": 1, "dim": 128, "page": 50, "k": 4, "sink": 0, "window": 256, "type": "bf16"},
        # the first tokens of one small fp32 request: latency alone
        {"name": "attend-first-tokens", "op": "attend", "requests": 1, "longest": 61, "heads": 4, "group": 1, "dim": 64, "page": 64, "k": 0, "sink": 64, "window": 128, "type": "f32"},
        # retrieval decode at 128K: sink, 32 selected pages, a 4096-token window
        {"name": "attend-retrieval-128k", "op": "attend", "requests": 1, "longest": 131072, "heads": 8, "group": 4, "dim": 128, "page": 128, "k": 32, "sink": 128, "window": 4096, "type": "bf16"},
        # a ragged retrieval batch, one q head to a kv head, pages that end inside a strip
        {"name": "attend-landmark-b16", "op": "attend", "requests": 16, "longest": 32768, "heads": 32, "group": 1, "dim": 128, "page": 50, "k": 4, "sink": 0, "window": 256, "type": "bf16"},
        # a ragged batch that attends to all it holds (head size 100, eight q heads to a kv head)
        {"name": "attend-dense-ragged-64", "op": "attend", "requests": 64, "longest": 8192, "heads": 4, "group": 8, "dim": 100, "page": 16, "k": 0, "sink": 0, "window": 8192, "type": "f32"},
        # whole 128K contexts attended by four requests: the cache's bandwidth
        {"name": "attend-dense-128k-b4", "op": "attend", "requests": 4, "longest": 131072, "near": True, "heads": 8, "group": 4, "dim": 128, "page": 128, "k": 0, "sink": 0, "window": 131072, "type": "bf16"},
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))

    op = rng.choice(["tables", "append", "append", "select", "attend", "attend", "attend"])
    page = rng.choice([16, 24, 50, 64, 128] + [spread(8, 200)] * 5)
    if op == "tables":
        return {"op": op, "requests": spread(1, 512), "longest": spread(16, 32768), "page": page, "tokens": spread(1, 98304)}
    heads, group, dim = rng.choice([(4, 1, 64), (8, 4, 128), (32, 1, 128), (32, 1, 100), (4, 8, 128), (2, 5, 96), (8, 2, 64), (1, 16, 128)])
    kind = rng.choice(["bf16", "bf16", "f32"])
    if op == "append":
        most = 65536 // heads
        tokens = spread(1, most)
        return {"op": op, "tokens": tokens, "run": spread(1, tokens), "heads": heads, "dim": dim, "page": page, "type": kind}
    k, sink, window = spread(1, 64), rng.choice([0, 4, 64, 128]), rng.choice([1, 128, 256, 1000, 4096])
    if op == "select":  # more candidates than are kept
        longest = spread(sink + window + (2 * k + 3) * page, min(131072, 16384 * page))
        requests = spread(1, max(1, min(64, 2 ** 20 // (heads * longest))))
    else:
        requests = spread(1, 64)
        longest = spread(1, max(1, min(131072, 2 ** 21 // (heads * requests))))
    case = {"op": op, "requests": requests, "longest": longest, "heads": heads, "group": group, "dim": dim, "page": page,
            "k": k, "sink": sink, "window": window, "type": kind}
    if op == "attend" and rng.random() < 0.4:
        case["k"], case["window"] = 0, longest
    return case


def _lengths(case):
    """Tokens that each request holds: the first the longest, the others spread over (0, longest], a few empty where
    there are many; or all of nearly one length."""
    n, longest = case["requests"], case["longest"]
    if case.get("near"):
        return [longest - 1111 * r for r in range(n)]
    lens = [longest]
    for r in range(1, n):
        lens.append(0 if n >= 16 and r % 16 == 5 else 1 + int((longest - 1) * ((r * 0.6180339887) % 1.0)))
    return lens


def _new_lengths(case):
    """New tokens of each request of a tables case: `tokens` in all, uneven."""
    n, total = case["requests"], case["tokens"]
    if total < n:
        return [1 if r < total else 0 for r in range(n)]
    share = [1 + (7 * r) % 5 for r in range(n)]
    new = [total * s // sum(share) for s in share]
    new[0] += total - sum(new)
    return new


def _shape(case):
    p = 64 if case["dim"] <= 64 else 128
    g = p // 32
    strips = -(-case["page"] // STRIP)
    return p, g, strips, 16 * p + 64 * g


def _bounds(length, page, sink, window):
    """(sink end, first window token, first candidate page, candidates) of a request of `length` tokens."""
    full = length // page
    w0 = min(max(length - window, 0), full * page)
    end = min(sink, w0)
    first = sink // page
    return end, w0, first, max(0, min(-(-w0 // page), full) - first)


def work(case):
    if case["op"] == "tables":
        lens, new, page = _lengths(case), _new_lengths(case), case["page"]
        pages = sum(-(-(a + b) // page) - -(-a // page) for a, b in zip(lens, new))
        return {"bytes": 4.0 * (5 * len(lens) + case["tokens"] + 4 * pages), "flops": 0.0}
    p, g, strips, _ = _shape(case)
    size = 2 if case["type"] == "bf16" else 4
    if case["op"] == "append":
        rows = case["tokens"] * case["heads"]
        reps = sum(at % case["page"] == case["page"] - 1 for at in _places(case))
        return {"bytes": 2.0 * rows * (2 * size * case["dim"] + 2 * (p // 2 + 2 * g)) + 4.0 * reps * case["heads"] * p,
                "flops": 4.0 * rows * case["dim"]}
    q = case["requests"] * case["heads"] * case["group"] * case["dim"]
    if case["op"] == "select":
        cand = sum(_bounds(n, case["page"], case["sink"], case["window"])[3] for n in _lengths(case)) * case["heads"]
        return {"bytes": 4.0 * cand * p + size * q + 4.0 * case["requests"] * case["heads"] * case["k"], "flops": 2.0 * cand * p}
    rows = 0
    for n in _lengths(case):
        end, w0, first, count = _bounds(n, case["page"], case["sink"], case["window"])
        inner = min(case["k"], count) * case["page"]
        rows += min(n, end + (n - w0) + inner)
    rows *= case["heads"]
    return {"bytes": 2.0 * rows * (p // 2 + 2 * g) + (size + 4.0) * q, "flops": 4.0 * rows * case["group"] * case["dim"]}


# ---------------------------------------------------------------------------------------------
# the layout, in torch

def _codes(x, groups):
    """Codes (c + 8) and bf16 scales of rows x [..., P] in fp32."""
    x = x.unflatten(-1, (groups, 32))
    s = (x.abs().amax(-1) / x.new_full((1,), 7.0)).to(torch.bfloat16)  # a tensor: a plain number becomes a product
    s = torch.where(torch.isfinite(s), torch.where(s.float() < 2.0 ** -100, torch.zeros_like(s), s), torch.full_like(s, math.nan))
    inv = torch.where(s.float() > 0, 1.0 / s.float(), torch.zeros_like(s, dtype=torch.float32))
    c = torch.round(x * inv.unsqueeze(-1)).clamp(-7, 7).nan_to_num(0.0)
    return (c + 8).to(torch.uint8).flatten(-2), s


def _nibbles(codes):
    """Two codes to a byte, the even one low."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _k_words(codes, groups):
    """K codes [..., P] -> the row's bytes [..., P / 2] in the order of the strip."""
    return _nibbles(codes.unflatten(-1, (groups, 4, 8)).transpose(-3, -2).flatten(-3))


def _v_units(codes, groups):
    """V codes [..., P] -> the row's 16-bit units [..., lane 8, group] (int16)."""
    return _nibbles(codes.unflatten(-1, (groups, 8, 4)).transpose(-3, -2).flatten(-3)).view(torch.int16).unflatten(-1, (8, groups))


def _strips(k, v, groups):
    """Strips [..., bytes] of rows k, v [..., 16, P] in fp32."""
    kc, ks = _codes(k, groups)
    vc, vs = _codes(v, groups)
    kb = _k_words(kc, groups).flatten(-2)
    units = _v_units(vc, groups).unflatten(-3, (2, 4, 2))                      # [..., p, c, o, lane, g]
    vb = units.movedim(-2, -4).movedim(-2, -1).flatten(-5).contiguous().view(torch.uint8)  # [p, lane, c, g, o]
    sb = torch.cat([ks, vs], -1).flatten(-2).contiguous().view(torch.uint8)
    return torch.cat([kb, vb, sb], -1)


def _rows(strips, p, groups):
    """Rows k, v [..., 16, P] in fp32 that strips [..., bytes] hold."""
    def codes(b):
        return torch.stack([b & 15, b >> 4], -1).flatten(-2)

    kc = codes(strips[..., :8 * p]).unflatten(-1, (16, 4, groups, 8)).transpose(-3, -2).flatten(-3)
    vc = codes(strips[..., 8 * p:16 * p].contiguous().view(torch.int16).unflatten(-1, (2, 8, 4, groups, 2))
               .movedim(-1, -4).movedim(-2, -4).flatten(-5).contiguous().view(torch.uint8))
    vc = vc.unflatten(-1, (2, 4, 2, 8, groups, 4)).transpose(-3, -2).flatten(-3).flatten(-4, -2)
    s = strips[..., 16 * p:].contiguous().view(torch.bfloat16).unflatten(-1, (16, 2, groups)).float().repeat_interleave(32, -1)
    return (kc.float() - 8) * s[..., 0, :], (vc.float() - 8) * s[..., 1, :]


# ---------------------------------------------------------------------------------------------
# inputs

def _dtype(case):
    return torch.bfloat16 if case["type"] == "bf16" else torch.float32


def _places(case):
    """Rows of an append case, counted through its pages in order: runs of `run` consecutive tokens, each from a row
    inside its own first page."""
    page, run = case["page"], case["run"]
    places, base = [], 0
    for i in range(0, case["tokens"], run):
        n = min(run, case["tokens"] - i)
        at = (i // run * 37) % page
        places += range(base + at, base + at + n)
        base += -(-(at + n) // page) * page
    return places


def _keys(gen, shape, dim, gains):
    """Key or value rows, zero past `dim`: normal, a few channels larger than the others."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= gains
    x[..., dim:] = 0
    return x


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    page, op = case["page"], case["op"]
    st = {"case": case}
    if op == "tables":
        heads, dim, kind = 1, 64, "bf16"
        lens, new = _lengths(case), _new_lengths(case)
        total = [a + b for a, b in zip(lens, new)]
        held = [-(-a // page) for a in lens]
        need = sum(-(-t // page) for t in total)
        n_pages = need + 7
        max_pages = max(-(-t // page) for t in total) + 1
        order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
        st["new"] = torch.tensor(new, dtype=torch.int32, device="cuda")
    else:
        heads, dim, kind = case["heads"], case["dim"], case["type"]
        lens = [0] if op == "append" else _lengths(case)
        held = [-(-a // page) for a in lens]
        n_pages = max(1, _places(case)[-1] // page + 1 if op == "append" else sum(held))
        max_pages = max(1, max(held))
        order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    p = 64 if dim <= 64 else 128
    g, per = p // 32, -(-page // STRIP)
    if op == "tables":
        st["pool"] = torch.zeros((n_pages, heads, per, 16 * p + 64 * g), dtype=torch.uint8, device="cuda")
        st["rep"] = torch.zeros((n_pages, heads, p), device="cuda")
    else:
        gains = 0.5 + torch.rand((2, heads, 1, 1, p), generator=gen, device="cuda")
        gains[..., :: 37] *= 4.0
        st["rep"] = torch.zeros((n_pages, heads, p), device="cuda")
        st["pool"] = torch.zeros((n_pages, heads, per, 16 * p + 64 * g), dtype=torch.uint8, device="cuda")
        step = max(1, 2 ** 24 // (heads * per * 16 * p))
        for a in range(0, n_pages, step):
            n = min(step, n_pages - a)
            rows = [_keys(gen, (n, heads, per, 16, p), dim, gains[i]) for i in (0, 1)]
            if op != "select":
                st["pool"][a:a + n] = _strips(rows[0], rows[1], g)
            st["rep"][a:a + n] = rows[0].mean((2, 3))
    table = torch.full((len(lens), max_pages), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, h in enumerate(held):
        table[r, :h] = order[at:at + h]
        at += h
    st["table"], st["free"] = table, torch.cat([order[at:], order[:at]])
    st["n_free"] = torch.tensor([n_pages - at], dtype=torch.int32, device="cuda")
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["sizes"] = {"heads": heads, "dim": dim, "p": p, "g": g, "n_pages": n_pages, "max_pages": max_pages}
    if op == "tables":
        st["keep"] = st["lens"].clone()
    elif op == "append":
        at = torch.tensor(_places(case), dtype=torch.int64, device="cuda")
        st["slots"] = (order[at // page].long() * page + at % page).to(torch.int32)
        # the new rows are slices of one projection's output, as a fused product leaves them
        new = torch.randn((case["tokens"], 2, heads, dim), generator=gen, device="cuda") * gains[:, :, 0, 0, :dim]
        new = new.to(_dtype(case))
        st["k"], st["v"] = new[:, 0], new[:, 1]
    else:
        q = torch.randn((len(lens), heads * case["group"], dim), generator=gen, device="cuda")
        st["q"] = q.to(_dtype(case))
    if op == "attend" and case["k"]:
        idx = torch.full((len(lens), heads, case["k"]), -1, dtype=torch.int32, device="cuda")
        for r, n in enumerate(lens):
            _, _, first, count = _bounds(n, page, case["sink"], case["window"])
            k = min(case["k"], count)
            if k:
                pick = torch.rand((heads, count), generator=gen, device="cuda").argsort(-1)[:, :k]
                idx[r, :, :k] = (first + pick.sort(-1).values).to(torch.int32)
        st["idx"] = idx
    elif op == "attend":
        st["idx"] = None
    if own:
        import retrieval_block_sparse_b200 as rba
        st["store"] = rba.PagedStore(
            n_q_heads=heads * case.get("group", 1), n_kv_heads=heads, head_dim=dim, page_size=page, n_pages=n_pages,
            max_requests=len(lens), max_pages=max_pages, dtype=kind, pool=st["pool"], rep=st["rep"], table=st["table"],
            lens=st["lens"], free=st["free"], n_free=st["n_free"])
        if op == "attend":
            st["workspace"] = st["store"].attend_workspace()
        elif op == "select":
            st["workspace"] = st["store"].select_workspace()
    return st


# ---------------------------------------------------------------------------------------------
# the operators

def run(state):
    return {"tables": _tables, "append": _append, "select": _select, "attend": _attend}[state["case"]["op"]](state)


def _tables(st):
    """Tables grown by each request's new tokens, then cut back to the lengths to keep (rejected drafts)."""
    case = st["case"]
    if own:
        slots, starts = st["store"].extend(st["new"], case["tokens"])
        st["store"].truncate(st["keep"])
    else:
        slots, starts = _extend(st, case["tokens"])
        _truncate(st)
    return {"slots": slots, "starts": starts, "table": st["table"], "lens": st["lens"], "free": st["free"], "n_free": st["n_free"]}


def _extend(st, n_slots):
    page, lens, new, table = st["case"]["page"], st["lens"].long(), st["new"].long(), st["table"]
    starts = torch.cat([new.new_zeros(1), new.cumsum(0)])
    i = torch.arange(n_slots, device="cuda")
    r = torch.searchsorted(starts[1:], i, right=True).clamp(max=len(lens) - 1)
    live = i < starts[-1]
    pos = lens[r] + i - starts[r]
    held = (lens + page - 1) // page
    need = (lens + new + page - 1) // page - held
    j = pos // page
    fresh = j >= held[r]
    nth = (need.cumsum(0) - need)[r] + j - held[r]
    got = torch.where(fresh, st["free"][(st["n_free"] - 1 - nth).clamp(min=0)], table[r, j.clamp(max=table.shape[1] - 1)])
    first = live & fresh & (pos % page == 0)
    table[r[first], j[first]] = got[first]
    st["lens"] += st["new"]
    st["n_free"] -= need.sum().to(torch.int32)
    return torch.where(live, got * page + pos % page, -torch.ones_like(pos)).to(torch.int32), starts.to(torch.int32)


def _truncate(st):
    page, lens = st["case"]["page"], st["lens"].long()
    kept = torch.minimum(lens, st["keep"].long())
    held = (kept + page - 1) // page
    freed = ((lens + page - 1) // page - held).cumsum(0)
    n = torch.arange(len(st["free"]), device="cuda")
    r = torch.searchsorted(freed, n, right=True).clamp(max=len(lens) - 1)
    before = torch.cat([freed.new_zeros(1), freed])[r]
    back = n < freed[-1]
    pages = st["table"][r[back], (held[r] + n - before)[back]]
    st["free"][(st["n_free"] + freed[-1] - 1 - n)[back]] = pages
    st["n_free"] += freed[-1].to(torch.int32)
    st["lens"].copy_(kept)


def _append(st):
    """New rows written in 4 bits with the means of the pages they complete, and read back as the cache holds them."""
    if own:
        st["store"].append(st["slots"], st["k"], st["v"])
        k, v = st["store"].read(st["slots"])
        return {"k": k, "v": v, "rep": st["rep"]}
    z, page = st["sizes"], st["case"]["page"]
    p, g, pool = z["p"], z["g"], st["pool"]
    slots = st["slots"].long()
    at, row = slots // page, slots % page
    strip, t = row // STRIP, row % STRIP
    k, v = (torch.nn.functional.pad(x.float(), (0, p - z["dim"])) for x in (st["k"], st["v"]))
    (kc, ks), (vc, vs) = _codes(k, g), _codes(v, g)
    pool[..., :8 * p].unflatten(-1, (16, p // 2))[at, :, strip, t] = _k_words(kc, g)
    units = pool.view(torch.int16)[..., 4 * p:8 * p].unflatten(-1, (2, 8, 4, g, 2))
    units[at, :, strip, t // 8, :, t % 8 // 2, :, t % 2] = _v_units(vc, g)
    pool.view(torch.bfloat16)[..., 8 * p:].unflatten(-1, (16, 2 * g))[at, :, strip, t] = torch.cat([ks, vs], -1)
    done = at[row == page - 1]
    keys = _rows(pool[done], p, g)[0].flatten(-3, -2)[..., :page, :]
    st["rep"][done] = keys.mean(-2)
    keys, values = (x[torch.arange(len(t), device="cuda"), :, t, :z["dim"]] for x in _rows(pool[at, :, strip], p, g))
    return {"k": keys.to(st["k"].dtype), "v": values.to(st["v"].dtype), "rep": st["rep"]}


def _ranges(st):
    """(sink end, first window token, first candidate page, candidates) of every request."""
    case, lens = st["case"], st["lens"].long()
    full = lens // case["page"]
    w0 = torch.minimum((lens - case["window"]).clamp(min=0), full * case["page"])
    first = case["sink"] // case["page"]
    count = (torch.minimum(-(-w0 // case["page"]), full) - first).clamp(min=0)
    return w0.clamp(max=case["sink"]), w0, first, count


def _select(st):
    """The k best full pages of each (request, kv head) by the group's summed query; -1 where a request has fewer."""
    case, z = st["case"], st["sizes"]
    if own:
        return st["store"].select(st["q"], case["k"], case["sink"], case["window"], workspace=st["workspace"])
    _, _, first, count = _ranges(st)
    q = torch.nn.functional.pad(st["q"].double().unflatten(1, (z["heads"], case["group"])).sum(2), (0, z["p"] - z["dim"]))
    pages = st["table"][:, first:].clamp(min=0).long()
    scores = torch.einsum("rhp,rjhp->rhj", q, st["rep"][pages].double()).float()
    live = torch.arange(pages.shape[1], device="cuda") < count[:, None]
    scores = torch.where(live[:, None], scores, torch.full_like(scores, -math.inf))
    scores = torch.nn.functional.pad(scores, (0, max(0, case["k"] - scores.shape[-1])), value=-math.inf)
    best = scores.sort(dim=-1, descending=True, stable=True).indices[..., :case["k"]]
    none = torch.arange(case["k"], device="cuda") >= count[:, None, None]
    best = best.masked_fill(none, 2 ** 30).sort(-1).values
    return (best + first).masked_fill(none, -1).to(torch.int32)


def _attend(st):
    """Attention of one token of each request over its sink tokens, selected pages and window."""
    case, z = st["case"], st["sizes"]
    scale = 1.0 / math.sqrt(z["dim"])
    if own:
        return st["store"].attend(st["q"], st["idx"], case["sink"], case["window"], scale=scale, workspace=st["workspace"])
    page, heads, n = case["page"], z["heads"], case["requests"]
    lens = st["lens"].long()
    end, w0, first, count = _ranges(st)
    longest = case["longest"]
    window = torch.arange(min(z["max_pages"], -(-(case["window"] + page) // page) + 1), device="cuda")
    lists = [((w0 // page)[:, None] + window).unsqueeze(1).expand(n, heads, -1)]
    lows, highs = [w0], [lens]
    if case["sink"]:
        sink = torch.arange(min(z["max_pages"], -(-min(case["sink"], longest) // page)), device="cuda")
        lists.append(sink.expand(n, heads, -1))
        lows.append(torch.zeros_like(end))
        highs.append(end)
    if case["k"]:
        lists.append(st["idx"].long())
        lows.append(end)
        highs.append(w0)
    lo, hi = (torch.cat([b[:, None, None].expand(*x.shape) for b, x in zip(bs, lists)], -1) for bs in (lows, highs))
    j = torch.cat(lists, -1)                                                     # [request, head, page of the list]
    inside = (j >= 0) & (j < z["max_pages"])
    at = st["table"][torch.arange(n, device="cuda")[:, None, None], j.clamp(0, z["max_pages"] - 1)].long()
    strips = st["pool"][at.clamp(min=0), torch.arange(heads, device="cuda")[:, None]]
    k, v = _rows(strips, z["p"], z["g"])                                         # [r, h, page, strip, 16, P]
    pos = (j * page)[..., None] + torch.arange(k.shape[3] * 16, device="cuda")
    seen = inside[..., None] & (at >= 0)[..., None] & (pos >= lo[..., None]) & (pos < hi[..., None]) & (pos < (j * page + page)[..., None])
    seen = seen.flatten(2)
    k, v = (x.flatten(2, 4)[..., :z["dim"]].masked_fill(~seen[..., None], 0.0) for x in (k, v))
    q = st["q"].float().unflatten(1, (heads, case["group"]))
    x = torch.matmul(q * scale, k.transpose(-1, -2)).masked_fill(~seen[:, :, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)
    w = torch.exp(x - top)
    total = w.sum(-1, keepdim=True)
    out = torch.matmul(w, v) / total.clamp(min=torch.finfo(torch.float32).tiny)
    lse = torch.log(total) + top
    return out.flatten(1, 2), torch.where(total > 0, lse, torch.full_like(lse, -math.inf)).flatten(1)


# ---------------------------------------------------------------------------------------------
# from the definitions, in 64 bits

def _quantised(x, dim):
    """Values in 64 bits that rows x [..., dim] are held as: each group of 32 dims by its own scale."""
    out = torch.zeros_like(x, dtype=torch.float64)
    for a in range(0, dim, 32):
        part = x[..., a:a + 32].double()
        s = (part.abs().max(-1, keepdim=True).values / 7).float().to(torch.bfloat16).double()
        inv = (1 / s).float().double()  # the code is that of x times the scale's reciprocal, both rounded to 32 bits
        out[..., a:a + 32] = torch.where(s > 0, (part * inv).float().double().round().clamp(-7, 7) * s, torch.zeros_like(part))
    return out


def _value(strips, token, dims, p, which):
    """Values in 64 bits of one token's dims in strips [..., bytes], byte by byte from the layout."""
    g = p // 32
    group = dims // 32
    if which == 0:
        byte = token * (p // 2) + (dims % 32 // 8 * g + group) * 4 + dims % 8 // 2
    else:
        lane, c = dims % 32 // 4, token % 8 // 2
        byte = 8 * p + (((token // 8 * 8 + lane) * 4 + c) * 2 * g + 2 * group + token % 2) * 2 + dims % 4 // 2
    code = (strips[..., byte].long() >> (4 * (dims % 2))) & 15
    at = 16 * p + token * 4 * g + 2 * (which * g + group)
    bits = strips[..., at].long() + 256 * strips[..., at + 1].long()
    return (code - 8).double() * (bits << 16).to(torch.int32).view(torch.float32).double()


def exact(case, seed):
    if case["op"] in ("tables", "select"):
        return None
    st = prepare(case, seed)
    z, page = st["sizes"], case["page"]
    p, dim, per = z["p"], z["dim"], -(-page // STRIP)
    dims = torch.arange(p, device="cuda")
    if case["op"] == "append":
        slots = st["slots"].tolist()
        k, v = _quantised(st["k"], dim), _quantised(st["v"], dim)
        rep, now = st["rep"].double(), {s: i for i, s in enumerate(slots)}
        for s in slots:
            if s % page == page - 1:
                a = s // page
                held = torch.stack([_value(st["pool"][a, :, t // 16], t % 16, dims, p, 0) for t in range(page)])
                mine = [t for t in range(page) if a * page + t in now]
                held[mine] = torch.nn.functional.pad(k[[now[a * page + t] for t in mine]], (0, p - dim))
                rep[a] = held.mean(0)
        return {"k": k, "v": v, "rep": rep}
    outs, lses = [], []
    for r, n in enumerate(st["lens"].tolist()):
        end, w0, _, _ = _bounds(n, page, case["sink"], case["window"])
        if n == 0:
            outs.append(torch.zeros((z["heads"], case["group"], dim), dtype=torch.float64, device="cuda"))
            lses.append(torch.full((z["heads"], case["group"]), -math.inf, dtype=torch.float64, device="cuda"))
            continue
        pages = -(-n // page)
        t = torch.arange(pages * page, device="cuda")
        seen = ((t < end) | ((t >= w0) & (t < n))).expand(z["heads"], -1).clone()
        if case["k"]:
            chosen = torch.zeros((z["heads"], pages + 1), dtype=torch.bool, device="cuda")
            picks = st["idx"][r].long()
            chosen.scatter_(1, torch.where(picks < 0, pages, picks), True)
            seen |= chosen[:, :pages].repeat_interleave(page, 1) & (t >= end) & (t < w0)
        keys = []
        for which in (0, 1):
            x = torch.zeros((z["heads"], pages, per * 16, dim), dtype=torch.float64, device="cuda")
            for s in range(per):
                strips = st["pool"][st["table"][r, :pages].long(), :, s]
                for i in range(16):
                    x[:, :, s * 16 + i] = _value(strips, i, dims[:dim], p, which).transpose(0, 1)
            keys.append(x[:, :, :page].flatten(1, 2))
        q = st["q"][r].double().view(z["heads"], case["group"], dim)
        logits = torch.einsum("hgd,htd->hgt", q, keys[0]) / math.sqrt(dim)
        logits.masked_fill_(~seen[:, None], -math.inf)
        lses.append(torch.logsumexp(logits, -1))
        outs.append(torch.einsum("hgt,htd->hgd", torch.softmax(logits, -1), keys[1]))
        del keys, logits
    return torch.stack(outs).flatten(1, 2), torch.stack(lses).flatten(1)
