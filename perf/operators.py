"""The paged-cache operators: listed workloads, drawn ones, and plain forms.

Four operators over one cache of pages in E4M3 with a scale for each page and
head: the page tables (``tables``), the write of new keys and values
(``append``), the score of each page for a query (``scores``) and the attention
(``decode``; over whole tables, or over the pages a list selects).

A case is a dict of plain values. ``prepare`` makes its inputs from a seed,
``run`` makes one pass: the library's call where ``own`` is true, else the same
result from elementary torch operations in 32 bits. ``exact`` computes it in 64
bits, written apart from both.
"""
import math
import random

import torch

own = False

DEV = "cuda"
MIN_SCALE = 2.0 ** -120  # the scale of a page that holds nothing but zeros


def listed():
    return [
        # One token for each running request, some of which have just ended: the table update of a decode step.
        {"name": "tables-step", "op": "tables", "R": 96, "lo": 1, "hi": 32768, "new": 1, "ended": 5, "P": 64},
        # Prompts being admitted beside running requests, small pages.
        {"name": "tables-prompts", "op": "tables", "R": 700, "lo": 0, "hi": 8192, "new": 400, "ended": 20, "P": 16},
        # One new token for each request: most land inside a page that is partly filled.
        {"name": "append-step", "op": "append", "R": 96, "new": 1, "Hkv": 8, "D": 128, "P": 64, "layout": "heads"},
        # A few verify tokens each, odd counts, small heads, token-major pages.
        {"name": "append-verify", "op": "append", "R": 333, "new": 5, "Hkv": 5, "D": 64, "P": 16, "layout": "tokens"},
        # Chunks of prompts, keys and values as slices of one fused projection.
        {"name": "append-prompts", "op": "append", "R": 23, "new": 1425, "Hkv": 8, "D": 128, "P": 64, "layout": "heads"},
        # A small batch at ordinary lengths.
        {"name": "scores-step", "op": "scores", "R": 8, "G": 1, "lo": 1024, "hi": 8191, "Hq": 64, "Hkv": 8, "D": 128, "P": 64},
        # Long contexts with verify rows: where choosing pages pays.
        {"name": "scores-long", "op": "scores", "R": 48, "G": 2, "lo": 8192, "hi": 131072, "Hq": 64, "Hkv": 8, "D": 128, "P": 64},
        # One short request: the latency of a call.
        {"name": "decode-one", "op": "decode", "R": 1, "G": 1, "lo": 777, "hi": 777, "Hq": 32, "Hkv": 8, "D": 128, "P": 64, "layout": "heads", "K": 0},
        # Verify rows, a group of three, small pages and heads, odd lengths.
        {"name": "decode-verify", "op": "decode", "R": 31, "G": 4, "lo": 0, "hi": 5001, "Hq": 24, "Hkv": 8, "D": 64, "P": 16, "layout": "tokens", "K": 0},
        # An ordinary batch of mixed lengths.
        {"name": "decode-batch", "op": "decode", "R": 64, "G": 1, "lo": 1024, "hi": 8192, "Hq": 64, "Hkv": 8, "D": 128, "P": 64, "layout": "heads", "K": 0},
        # Long contexts, many query heads for each head of the cache, two verify rows.
        {"name": "decode-long", "op": "decode", "R": 16, "G": 2, "lo": 4096, "hi": 131072, "Hq": 128, "Hkv": 8, "D": 128, "P": 128, "layout": "heads", "K": 0},
        # The pages that a select chose out of long contexts.
        {"name": "decode-selected", "op": "decode", "R": 64, "G": 1, "lo": 16384, "hi": 65536, "Hq": 64, "Hkv": 8, "D": 128, "P": 64, "layout": "heads", "K": 64},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "scores", "decode", "decode"])
    P = rng.choice([16, 32, 64, 128])
    if op == "tables":
        return {"op": op, "R": _log(rng, 1, 2000), "lo": rng.choice([0, 1]), "hi": _log(rng, 16, 32768), "new": _log(rng, 1, 400),
                "ended": rng.choice([0, 3, 30]), "P": P}
    Hkv, D = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([64, 128, 128, 256])
    layout = rng.choice(["heads", "tokens"])
    if op == "append":
        R = _log(rng, 1, 400)
        return {"op": op, "R": R, "new": _log(rng, 1, max(1, 32768 // R)), "Hkv": Hkv, "D": D, "P": P, "layout": layout}
    g = rng.choice([1, 2, 3, 4, 7, 8, 16])
    G = rng.choice([1, 1, 2, 4])
    R = _log(rng, 1, 128)
    if op == "scores":
        hi = _log(rng, 64, min(131072, (1 << 31) // (R * Hkv * D)))
        return {"op": op, "R": R, "G": G, "lo": rng.randint(0, hi), "hi": hi, "Hq": g * Hkv, "Hkv": Hkv, "D": D, "P": P}
    hi = _log(rng, 1, min(131072, (1 << 29) // (R * Hkv * D)))
    K = rng.choice([0, 0, max(1, hi // P // 5)])
    return {"op": op, "R": R, "G": G, "lo": rng.randint(0, hi), "hi": hi, "Hq": g * Hkv, "Hkv": Hkv, "D": D, "P": P, "layout": layout, "K": K}


# ---- inputs ---------------------------------------------------------------------------------------------------

def _lengths(c):
    """The requests' lengths go by the case alone, so that work() knows them; the first is the longest."""
    r = random.Random("lengths %(R)d %(lo)d %(hi)d" % c)
    return [c["hi"]] + [r.randint(c["lo"], c["hi"]) for _ in range(c["R"] - 1)]


def _news(c):
    """New tokens of each request (-1: the request has ended): one each, or up to twice `new`, the first the most."""
    r = random.Random("new %(R)d %(new)d" % c)
    n = [c["new"]] * c["R"] if c["new"] == 1 else [2 * c["new"]] + [r.randint(0, 2 * c["new"]) for _ in range(c["R"] - 1)]
    for i in range(min(c.get("ended", 0), c["R"] - 1)):
        n[1 + (i * 37) % (c["R"] - 1)] = -1
    return n


def _befores(c):
    """Tokens that the append's requests already have."""
    r = random.Random("before %(R)d %(P)d" % c)
    return [r.randint(0, 3 * c["P"]) for _ in range(c["R"])]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _two_to(e):
    """2^e in 32 bits, exactly (|e| <= 126)."""
    return ((e + 127) << 23).int().view(torch.float32)


def _scales(g, *shape):
    """Powers of two around 2^-7, as keys and values of about unit size give."""
    return _two_to(torch.randint(-9, -5, shape, generator=g, device=DEV))


def _codes(g, shape):
    """E4M3 codes of normally distributed values, filled in pieces."""
    out = torch.empty(shape, dtype=torch.uint8, device=DEV)
    flat = out.view(-1)
    step = 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        x = torch.randn(n, generator=g, device=DEV, dtype=torch.float32).mul_(90.0).clamp_(-448, 448)
        flat[i:i + n] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def _pages_of(codes, layout):
    """A pool as [pages, heads, tokens, D], whichever of heads and tokens lies further out in memory."""
    return codes if layout == "heads" else codes.transpose(1, 2)


def _pool(g, pages, c):
    shape = (pages, c["Hkv"], c["P"], c["D"]) if c["layout"] == "heads" else (pages, c["P"], c["Hkv"], c["D"])
    return _pages_of(_codes(g, shape), c["layout"])


def _table(g, lens, P, spare):
    """A table of pages in random order; entries past a request's length hold any page."""
    need = torch.tensor([-(-n // P) for n in lens], device=DEV)
    W, total = max(1, int(need.max())), int(need.sum())
    pages = total + spare
    perm = torch.randperm(pages, generator=g, device=DEV)
    col = torch.arange(W, device=DEV)
    at = (need.cumsum(0) - need)[:, None] + col
    return torch.where(col < need[:, None], perm[at.clamp(max=pages - 1)], perm[0]).int(), pages


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "tables":
        P, lens, new = c["P"], _lengths(c), _news(c)
        W = max(-(-(a + max(0, b)) // P) for a, b in zip(lens, new))
        held = sum(-(-n // P) for n in lens)
        wanted = sum(max(0, -(-(a + b) // P) - -(-a // P)) for a, b in zip(lens, new) if b >= 0)
        table, pages = _table(g, lens, P, wanted + 64)
        table = torch.cat([table, torch.zeros(c["R"], W - table.shape[1], dtype=torch.int32, device=DEV)], 1).contiguous()
        used = torch.zeros(pages, dtype=torch.bool, device=DEV)
        col = torch.arange(W, device=DEV)
        used[table[col < torch.tensor([-(-n // P) for n in lens], device=DEV)[:, None]].long()] = True
        free = torch.nonzero(~used).view(-1)
        free = free[torch.randperm(len(free), generator=g, device=DEV)].int()
        taken = int(torch.randint(0, pages, (1,), generator=g, device=DEV))
        ring = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
        ring[(taken + torch.arange(len(free), device=DEV)) % pages] = free
        s |= {"lengths": _i32(lens), "new": _i32(new), "table": table, "ring": ring,
              "state": torch.tensor([taken, taken + len(free)], dtype=torch.int64, device=DEV),
              "T": sum(max(0, n) for n in new) + 7}
        assert len(free) == pages - held
        return s
    P, D, Hkv = c["P"], c["D"], c["Hkv"]
    if c["op"] == "append":
        before, new = _befores(c), _news(c)
        table, pages = _table(g, [a + b for a, b in zip(before, new)], P, 5)
        at = [(r, a + i) for r, (a, b) in enumerate(zip(before, new)) for i in range(b)]
        req, pos = (torch.tensor(v, device=DEV) for v in zip(*at))
        s["slots"] = (table[req, pos // P] * P + pos % P).int()
        T = len(at)
        fused = torch.randn(T, (c["Hkv"] * 3) * D, generator=g, device=DEV)  # queries, keys and values of a layer
        fused = (fused * _two_to(torch.randint(-3, 4, (T, 1), generator=g, device=DEV))).bfloat16()
        s["k"] = fused[:, Hkv * D:2 * Hkv * D].view(T, Hkv, D)
        s["v"] = fused[:, 2 * Hkv * D:].view(T, Hkv, D)
        s["k_pool"], s["v_pool"] = _pool(g, pages, c), _pool(g, pages, c)
        s["k_scale"], s["v_scale"] = _scales(g, pages, Hkv), _scales(g, pages, Hkv)
        b = torch.randn(pages, Hkv, 2, D, generator=g, device=DEV)
        s["bounds"] = torch.stack([b.amax(2), b.amin(2)], 2).bfloat16()
        return s
    lens = _lengths(c)
    table, pages = _table(g, lens, P, 5)
    s |= {"table": table, "lengths": _i32(lens), "q": torch.randn(c["R"] * c["G"], c["Hq"], D, generator=g, device=DEV).bfloat16()}
    if c["op"] == "scores":
        hi = torch.randn(pages, Hkv, D, generator=g, device=DEV).abs() + 1.5  # about the extremes of a page of normal keys
        lo = -(torch.randn(pages, Hkv, D, generator=g, device=DEV).abs() + 1.5)
        s["bounds"] = torch.stack([hi, lo], 2).bfloat16()
        return s
    s["k_pool"], s["v_pool"] = _pool(g, pages, c), _pool(g, pages, c)
    s["k_scale"], s["v_scale"] = _scales(g, pages, Hkv), _scales(g, pages, Hkv)
    if c["K"]:
        # As the select leaves them: ascending, with -1 past a row's count.
        B, W, K = c["R"] * c["G"], table.shape[1], c["K"]
        have = torch.tensor([-(-n // P) for n in lens], device=DEV).repeat_interleave(c["G"])[:, None, None]
        score = torch.rand(B, Hkv, W, generator=g, device=DEV).masked_fill(torch.arange(W, device=DEV) >= have, -1.0)
        top = score.topk(min(K, W), -1).indices
        lists = torch.where(top < have, top, W).sort(-1).values
        s["counts"] = (lists < W).sum(-1).int()
        s["lists"] = torch.where(lists < W, lists, -1).int().contiguous()
    return s


# ---- one pass ---------------------------------------------------------------------------------------------------

def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _own_tables(s):
    from sparse_mla_decode_gb300 import binding
    if "out" not in s:
        R = s["lengths"].numel()
        s["out"] = {k: torch.empty(n, dtype=t, device=DEV) for k, n, t in (
            ("new_lengths", R, torch.int32), ("new_state", 2, torch.int64), ("starts", R + 1, torch.int32),
            ("slots", s["T"], torch.int32), ("positions", s["T"], torch.int32))}
    binding.block_tables(s["lengths"], s["new"], s["table"], s["ring"], s["state"], s["case"]["P"], **s["out"])
    return {"table": s["table"], "ring": s["ring"], **s["out"]}


def _cache(s):
    from sparse_mla_decode_gb300 import binding
    if "cache" not in s:
        s["cache"] = binding.PagedCache(s.get("k_pool"), s.get("v_pool"), s.get("k_scale"), s.get("v_scale"), s.get("bounds"), page_size=s["case"]["P"])
    return s["cache"]


def _own_append(s):
    from sparse_mla_decode_gb300 import binding
    binding.paged_append(_cache(s), s["k"], s["v"], s["slots"])
    return _pools(s)


def _own_scores(s):
    from sparse_mla_decode_gb300 import binding
    if "out" not in s:
        s["out"] = torch.empty(s["q"].shape[0], s["case"]["Hkv"], s["table"].shape[1], dtype=torch.bfloat16, device=DEV)
    return binding.block_scores(s["q"], _cache(s), s["table"], s["lengths"], row_group=s["case"]["G"], keep_first=1, keep_last=2, out=s["out"])


def _own_decode(s):
    from sparse_mla_decode_gb300 import binding
    c, q = s["case"], s["q"]
    if "out" not in s:
        s["out"], s["lse"] = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float32, device=DEV)
        s["workspace"] = torch.zeros(binding.paged_workspace_bytes(_cache(s)), dtype=torch.uint8, device=DEV)
    out, lse = binding.paged_decode(q, _cache(s), s["table"], s["lengths"], c["D"] ** -0.5, row_group=c["G"], block_lists=s.get("lists"),
                                    block_counts=s.get("counts"), out=s["out"], lse=s["lse"], workspace=s["workspace"])
    return {"out": out, "lse": lse}


_own = {"tables": _own_tables, "append": _own_append, "scores": _own_scores, "decode": _own_decode}


def _pools(s):
    f8 = torch.float8_e4m3fn
    return {"k": s["k_pool"].view(f8), "v": s["v_pool"].view(f8), "k_scale": s["k_scale"], "v_scale": s["v_scale"], "bounds": s["bounds"]}


def _before(x):
    return x.cumsum(0) - x


def _plain_tables(s):
    P, T = s["case"]["P"], s["T"]
    length, new, table, ring = s["lengths"].long(), s["new"].long(), s["table"], s["ring"]
    R, W = table.shape
    pages, taken, given = ring.numel(), s["state"][0], s["state"][1]
    have, want = (length + P - 1) // P, new.clamp(min=0)
    want = want * ((length + want + P - 1) // P <= W)
    need = (length + want + P - 1) // P - have
    off = _before(need)
    want = want * ((need == 0) | (off + need <= given - taken))
    want = want * (_before(want) + want <= T)
    need = need * (want > 0)
    starts = torch.cat([want.new_zeros(1), want.cumsum(0)])
    col = torch.arange(W, device=DEV)
    fresh = ring[(taken + off[:, None] + col - have[:, None]) % pages]
    taking = (col >= have[:, None]) & (col < (have + need)[:, None])
    full = torch.where(taking, fresh, table)
    back = have.clamp(max=W) * (new < 0)
    put = torch.where(col < back[:, None], (given + _before(back)[:, None] + col) % pages, pages)
    ring = torch.cat([ring, ring.new_zeros(1)]).scatter(0, put.view(-1), table.reshape(-1))[:pages]
    t = torch.arange(T, device=DEV)
    r = torch.searchsorted(starts[1:].contiguous(), t, right=True).clamp(max=R - 1)
    pos = length[r] + t - starts[r]
    live = t < starts[-1]
    page = full[r, (pos // P).clamp(max=W - 1)].long()
    return {"table": full, "ring": ring, "new_lengths": torch.where(new < 0, 0, length + want).int(),
            "new_state": torch.stack([taken + need.sum(), given + back.sum()]), "starts": starts.int(),
            "slots": torch.where(live, page * P + pos % P, -1).int(), "positions": torch.where(live, pos, -1).int()}


def _power(amax):
    """The least power of two at which amax / power is at most 448."""
    m, e = torch.frexp(amax.clamp(min=2.0 ** -126))
    return _two_to((e - 9 + (m > 0.875)).clamp(-120, 120))


def _over_pages(start, at, x, how):
    """The extremes of x's rows over the rows of each page, from `start` on."""
    return start.scatter_reduce(0, at.view(-1, *[1] * (x.dim() - 1)).expand_as(x), x, how)


def _plain_append(s):
    P, slots = s["case"]["P"], s["slots"].long()
    touched, at = torch.unique(slots // P, return_inverse=True)
    offset, n = slots % P, touched.numel()
    first = torch.full((n,), P, device=DEV).scatter_reduce(0, at, offset, "amin")
    kept = torch.arange(P, device=DEV) < first[:, None]
    for x, pool, scale in ((s["k"], s["k_pool"], s["k_scale"]), (s["v"], s["v_pool"], s["v_scale"])):
        x = x.float()
        size = _over_pages(torch.zeros(n, x.shape[1], device=DEV), at, x.abs().amax(-1), "amax")
        was = torch.where(first[:, None] > 0, scale[touched], MIN_SCALE)
        now = torch.maximum(was, _power(size))
        old = pool[touched].view(torch.float8_e4m3fn).float()
        again = (old * (was / now)[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        page = torch.where(kept[:, None, :, None], again, pool[touched])
        page[at, :, offset] = (x / now[at][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        pool[touched], scale[touched] = page, now
    k = s["k"].float()
    inf = torch.full((n, *k.shape[1:]), math.inf, device=DEV)
    was = s["bounds"][touched].float()
    part = (first > 0)[:, None, None]
    hi = _over_pages(torch.where(part, was[:, :, 0], -inf), at, k, "amax")
    lo = _over_pages(torch.where(part, was[:, :, 1], inf), at, k, "amin")
    s["bounds"][touched] = torch.stack([hi, lo], 2).bfloat16()
    return _pools(s)


def _limits(s):
    """The tokens that each row sees: verify row i of G sees the first length - G + 1 + i."""
    G = s["case"]["G"]
    return (s["lengths"].long()[:, None] - G + 1 + torch.arange(G, device=DEV)).clamp(min=0)


def _plain_scores(s):
    c = s["case"]
    P, g = c["P"], c["Hq"] // c["Hkv"]
    b = s["bounds"][s["table"].long()].float()  # [R, W, Hkv, 2, D]
    q = s["q"].float().view(c["R"], c["G"], c["Hkv"], g, c["D"])
    hi, lo = b[:, :, :, 0].permute(0, 2, 3, 1), b[:, :, :, 1].permute(0, 2, 3, 1)  # [R, Hkv, D, W]
    up = torch.matmul(q.clamp(min=0).transpose(1, 2).flatten(2, 3), hi) + torch.matmul(q.clamp(max=0).transpose(1, 2).flatten(2, 3), lo)
    up = up.view(c["R"], c["Hkv"], c["G"], g, -1).amax(3).transpose(1, 2)  # [R, G, Hkv, W]
    have = ((_limits(s) + P - 1) // P)[:, :, None, None]
    col = torch.arange(up.shape[-1], device=DEV)
    up = up.masked_fill((col < 1) | (col >= have - 2), math.inf).masked_fill(col >= have, math.nan)
    return up.flatten(0, 1).bfloat16()


def _softmax_of(s, logits, v):
    """Rows of logits (masked: -inf) over values: the output and the natural logarithm of the sum; nothing seen: 0 and -inf."""
    m = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - m.masked_fill(m == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / total.masked_fill(total == 0, 1.0)
    return out, (m + torch.log(total)).squeeze(-1)


def _values(pool, scale, *at):
    return pool[at].view(torch.float8_e4m3fn).float().mul_(scale[at][..., None, None])


def _plain_decode(s):
    c = s["case"]
    R, G, Hkv, g, P, D = c["R"], c["G"], c["Hkv"], c["Hq"] // c["Hkv"], c["P"], c["D"]
    q, table, lim = s["q"].float() * D ** -0.5, s["table"].long(), _limits(s)
    token = torch.arange(P, device=DEV)
    if c["K"]:
        lists = s["lists"].long()
        listed_ = torch.arange(lists.shape[-1], device=DEV) < s["counts"][:, :, None]
        pages = table.repeat_interleave(G, 0)[:, None].expand(-1, Hkv, -1).gather(2, lists.clamp(min=0))  # [B, Hkv, K]
        heads = torch.arange(Hkv, device=DEV)[None, :, None]
        seen = ((lists[..., None] * P + token < lim.view(-1)[:, None, None, None]) & listed_[..., None]).flatten(2)[:, :, None]
        k = _values(s["k_pool"], s["k_scale"], pages, heads).flatten(2, 3)
        logits = torch.matmul(q.view(-1, Hkv, g, D), k.transpose(-1, -2)).masked_fill(~seen, -math.inf)
        out, lse = _softmax_of(s, logits, _values(s["v_pool"], s["v_scale"], pages, heads).flatten(2, 3))
    else:
        gather = lambda pool, scale: _values(pool, scale, table).transpose(1, 2).flatten(2, 3)  # noqa: E731  [R, Hkv, W * P, D]
        rows = q.view(R, G, Hkv, g, D).transpose(1, 2).flatten(2, 3)
        at = torch.arange(table.shape[1] * P, device=DEV)
        seen = (at < lim[:, :, None]).repeat_interleave(g, 1)[:, None]  # [R, 1, G * g, W * P]
        logits = torch.matmul(rows, gather(s["k_pool"], s["k_scale"]).transpose(-1, -2)).masked_fill_(~seen, -math.inf)
        out, lse = _softmax_of(s, logits, gather(s["v_pool"], s["v_scale"]))
        out, lse = (x.view(R, Hkv, G, g, *x.shape[3:]).transpose(1, 2).flatten(0, 1) for x in (out, lse))
    return {"out": out.reshape(R * G, c["Hq"], D).bfloat16(), "lse": lse.reshape(R * G, c["Hq"])}


_plain = {"tables": _plain_tables, "append": _plain_append, "scores": _plain_scores, "decode": _plain_decode}


# ---- what a pass cannot do without ----------------------------------------------------------------------------

def work(case):
    c = case
    P = c["P"]
    up = lambda n: -(-max(0, n) // P)  # noqa: E731
    if c["op"] == "tables":
        lens, new = _lengths(c), _news(c)
        T = sum(max(0, n) for n in new) + 7
        moved = sum(up(a) if n < 0 else up(a + n) - up(a) for a, n in zip(lens, new))
        return {"bytes": 16 * c["R"] + 8 * T + 8 * moved, "flops": 0}
    D, Hkv = c["D"], c["Hkv"]
    if c["op"] == "append":
        new = _news(c)
        pages = sum(up(a + n) - a // P for a, n in zip(_befores(c), new) if n)
        return {"bytes": sum(new) * (4 + 6 * Hkv * D) + pages * Hkv * (8 + 4 * D), "flops": 0}
    lens, G, Hq = _lengths(c), c["G"], c["Hq"]
    if c["op"] == "scores":
        pages = sum(up(n) for n in lens)
        return {"bytes": pages * (4 + Hkv * 4 * D) + 2 * c["R"] * G * (Hq * D + Hkv * max(map(up, lens))), "flops": 4.0 * pages * G * Hq * D}
    io = c["R"] * G * Hq * (4 * D + 4)
    if c["K"]:
        tokens = sum(min(max(0, n - G + 1 + i), c["K"] * P) for n in lens for i in range(G))  # of each row and kv head
        return {"bytes": io + tokens * Hkv * 2 * D + -(-tokens // P) * Hkv * 16, "flops": 4.0 * tokens * Hq * D}
    return {"bytes": io + sum(lens) * Hkv * 2 * D + sum(map(up, lens)) * (4 + 8 * Hkv),
            "flops": 4.0 * D * Hq * sum(max(0, n - G + 1 + i) for n in lens for i in range(G))}


# ---- 64 bits --------------------------------------------------------------------------------------------------

def _e4m3_values():
    """The 256 values of E4M3 from its definition: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN."""
    v = []
    for b in range(128):
        e, m = b >> 3, b & 7
        v.append(math.nan if b == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return torch.tensor(v + [-x for x in v], dtype=torch.float64, device=DEV)


def _nearest_e4m3(x):
    """The value of E4M3 nearest to x (64 bits, |x| <= 448), ties to the even code."""
    v = _e4m3_values()[:127]
    a = x.abs()
    below = (torch.searchsorted(v, a.contiguous(), right=True) - 1).clamp(0, 126)
    above = (below + 1).clamp(max=126)
    d, u = a - v[below], v[above] - a
    near = torch.where((u < d) | ((u == d) & (above % 2 == 0)), above, below)
    return torch.copysign(v[near], x)


def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    return _exact_scores(s) if case["op"] == "scores" else _exact_decode(s)


def _exact_append(s):
    P, v = s["case"]["P"], _e4m3_values()
    slots = s["slots"].tolist()
    got = {"bounds": s["bounds"].double()}
    runs, i = [], 0
    for j in range(1, len(slots) + 1):
        if j == len(slots) or slots[j] // P != slots[i] // P:
            runs.append((slots[i] // P, slots[i] % P, i, j))
            i = j
    for n in "kv":
        x, pool, scale = s[n].double(), v[s[n + "_pool"].long()], s[n + "_scale"].double()
        for p, o, a, b in runs:
            m, e = torch.frexp(x[a:b].abs().amax((0, 2)) / 448)  # m * 2^e, 1/2 <= m < 1
            now = (torch.where(m > 0.5, e, e - 1).clamp(-120, 120).long() + 1023 << 52).view(torch.float64)
            if o:
                now = torch.maximum(now, scale[p])
                pool[p, :, :o] = _nearest_e4m3(pool[p, :, :o] * (scale[p] / now)[:, None, None])
            pool[p, :, o:o + b - a] = _nearest_e4m3(x[a:b].transpose(0, 1) / now[:, None, None])
            scale[p] = now
            if n == "k":
                y = x[a:b] if not o else torch.cat([x[a:b], got["bounds"][p].transpose(0, 1)])
                got["bounds"][p] = torch.stack([y.amax(0), y.amin(0)], 1)
        got |= {n: pool, n + "_scale": scale}
    return got


def _exact_scores(s):
    c, P = s["case"], s["case"]["P"]
    g, W = c["Hq"] // c["Hkv"], s["table"].shape[1]
    out = torch.full((c["R"] * c["G"], c["Hkv"], W), math.nan, dtype=torch.float64, device=DEV)
    for r, n in enumerate(s["lengths"].tolist()):
        for i in range(c["G"]):
            have = -(-max(0, n - c["G"] + 1 + i) // P)
            b = s["bounds"][s["table"][r, :have].long()].double()  # [have, Hkv, 2, D]
            q = s["q"][r * c["G"] + i].double().view(c["Hkv"], g, c["D"])
            row = out[r * c["G"] + i]
            for h in range(c["Hkv"]):
                for j in range(g):
                    up = torch.maximum(q[h, j] * b[:, h, 0], q[h, j] * b[:, h, 1]).sum(-1)
                    row[h, :have] = up if j == 0 else torch.maximum(row[h, :have], up)
            row[:, :min(1, have)] = math.inf
            row[:, max(0, have - 2):have] = math.inf
    return out


def _exact_decode(s):
    c, v = s["case"], _e4m3_values()
    G, Hkv, g, P, D = c["G"], c["Hkv"], c["Hq"] // c["Hkv"], c["P"], c["D"]
    out = torch.zeros(c["R"] * G, Hkv, g, D, dtype=torch.float64, device=DEV)
    lse = torch.full((c["R"] * G, Hkv, g), -math.inf, dtype=torch.float64, device=DEV)
    heads = torch.arange(Hkv, device=DEV)[:, None]
    for r, n in enumerate(s["lengths"].tolist()):
        if not n:
            continue
        for i in range(G):
            b, lim = r * G + i, max(0, n - G + 1 + i)
            if not lim:
                continue
            if c["K"] or i == 0:
                blocks = s["lists"][b].long().clamp(min=0) if c["K"] else torch.arange(-(-n // P), device=DEV).expand(Hkv, -1)
                pages = s["table"][r].long()[blocks]  # [Hkv, blocks]
                kv = [(v[s[x + "_pool"][pages, heads].long()] * s[x + "_scale"].double()[pages, heads][..., None, None]).flatten(1, 2) for x in "kv"]
                pos = (blocks[..., None] * P + torch.arange(P, device=DEV)).flatten(1)
            seen = pos < lim
            if c["K"]:
                seen = seen & (torch.arange(blocks.shape[1], device=DEV) < s["counts"][b][:, None]).repeat_interleave(P, 1)
            q = s["q"][b].double().view(Hkv, g, D)
            x = torch.einsum("hgd,hnd->hgn", q, kv[0]) / math.sqrt(D)
            x = x.masked_fill(~seen[:, None], -math.inf)
            lse[b] = torch.logsumexp(x, -1)
            out[b] = torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1), torch.where(seen[..., None], kv[1], 0.0))
    return {"out": out.view(c["R"] * G, c["Hq"], D), "lse": lse.view(c["R"] * G, c["Hq"])}
