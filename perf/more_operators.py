"""A speculative step over a paged cache in 4 bits: listed workloads, drawn ones, and plain forms.

Five operators, in the order of a step: the norm of each query and key head with the
position rotation in one pass, over one position axis or several (``rope``); the write of new
keys and values as E2M1 codes with an E4M3 scale for each 16 columns, and reading them back
(``append``); attention over that cache, whole tables or listed pages (``decode``); the
verification of drafted tokens against the target's probabilities (``verify``); and the pages
of rejected tokens, which go back to the ring of free ones (``trim``).

A case is a dict of plain values. ``prepare`` makes its inputs from a seed, ``run``
makes one pass: the library's call where ``own`` is true, else the same result from elementary
torch operations in 32 bits (64 where angles or sums need them). ``exact`` computes it
in 64 bits, written apart from both.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # of the E2M1 codes 0 to 7


def listed():
    return [
        # The queries and keys of a decode step, one token for each running request.
        {"name": "rope-step", "op": "rope", "T": 96, "Hq": 64, "Hkv": 8, "D": 128, "rot": 128, "axes": 1, "norm": True, "inter": False, "far": 131072},
        # Prompts with images and video among them: three position axes, slices of one fused projection.
        {"name": "rope-prompts", "op": "rope", "T": 28001, "Hq": 64, "Hkv": 8, "D": 128, "rot": 128, "axes": 3, "norm": True, "inter": False, "far": 32768},
        # One new token for each request.
        {"name": "append-step", "op": "append", "R": 96, "new": 1, "Hkv": 8, "D": 128, "P": 64, "layout": "heads"},
        # Chunks of prompts, keys and values as slices of one fused projection, odd lengths.
        {"name": "append-prompts", "op": "append", "R": 23, "new": 1425, "Hkv": 8, "D": 128, "P": 64, "layout": "heads"},
        # A few short requests with verify rows, a group of three, small pages and heads: latency.
        {"name": "decode-verify", "op": "decode", "R": 5, "G": 4, "lo": 0, "hi": 777, "Hq": 24, "Hkv": 8, "D": 64, "P": 16, "layout": "tokens", "K": 0},
        # An ordinary batch of mixed lengths.
        {"name": "decode-batch", "op": "decode", "R": 64, "G": 1, "lo": 1024, "hi": 8192, "Hq": 64, "Hkv": 8, "D": 128, "P": 64, "layout": "heads", "K": 0},
        # Long contexts, many query heads for each head of the cache, two verify rows.
        {"name": "decode-long", "op": "decode", "R": 16, "G": 2, "lo": 4096, "hi": 131072, "Hq": 128, "Hkv": 8, "D": 128, "P": 128, "layout": "heads", "K": 0},
        # The pages that a select chose out of long contexts.
        {"name": "decode-selected", "op": "decode", "R": 64, "G": 1, "lo": 16384, "hi": 65536, "Hq": 64, "Hkv": 8, "D": 128, "P": 64, "layout": "heads", "K": 64},
        # One request, three drafted tokens, an odd vocabulary: the latency of a call.
        {"name": "verify-one", "op": "verify", "R": 1, "G": 4, "V": 100003, "given": True},
        # A batch whose drafts come with their own distributions.
        {"name": "verify-batch", "op": "verify", "R": 96, "G": 6, "V": 131072, "given": True},
        # After the verification of a batch: a few tokens off the end of each request.
        {"name": "trim-step", "op": "trim", "R": 96, "lo": 1, "hi": 32768, "drop": 7, "P": 64},
        # Many requests taken back to a common beginning, small pages.
        {"name": "trim-far", "op": "trim", "R": 2000, "lo": 0, "hi": 8192, "drop": 8192, "P": 16},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "decode", "verify", "trim"])
    P = rng.choice([16, 32, 64, 128])
    Hkv, D = rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([64, 128, 128, 256])
    g = rng.choice([1, 2, 3, 4, 7, 8, 16])
    layout = rng.choice(["heads", "tokens"])
    if op == "rope":
        return {"op": op, "T": _log(rng, 1, min(28000, (1 << 28) // ((g + 1) * Hkv * D))), "Hq": g * Hkv, "Hkv": Hkv, "D": D, "rot": rng.choice([D, D, D // 2, 16, 48]),
                "axes": rng.choice([1, 1, 2, 3, 4]), "norm": rng.choice([True, True, False]), "inter": rng.choice([False, False, True]), "far": _log(rng, 16, 1 << 20)}
    if op == "append":
        R = _log(rng, 1, 400)
        return {"op": op, "R": R, "new": _log(rng, 1, max(1, 32768 // R)), "Hkv": Hkv, "D": D, "P": P, "layout": layout}
    if op == "verify":
        R, G = _log(rng, 1, 128), rng.choice([1, 2, 3, 4, 6, 8])
        return {"op": op, "R": R, "G": G, "V": _log(rng, 2, min(200000, 80_000_000 // (R * G))), "given": rng.choice([True, True, False])}
    if op == "trim":
        return {"op": op, "R": _log(rng, 1, 2000), "lo": rng.choice([0, 1]), "hi": _log(rng, 16, 32768), "drop": _log(rng, 1, 4096), "P": P}
    G = rng.choice([1, 1, 2, 4])
    R = _log(rng, 1, 128)
    hi = _log(rng, 1, min(131072, (1 << 29) // (R * Hkv * D)))
    K = rng.choice([0, 0, max(1, hi // P // 5)])
    return {"op": op, "R": R, "G": G, "lo": rng.randint(0, hi), "hi": hi, "Hq": g * Hkv, "Hkv": Hkv, "D": D, "P": P, "layout": layout, "K": K}


# ---- inputs ---------------------------------------------------------------------------------------------------

def _lengths(c):
    """The requests' lengths go by the case alone, so that work() knows them; the first is the longest."""
    r = random.Random("lengths %(R)d %(lo)d %(hi)d" % c)
    return [c["hi"]] + [r.randint(c["lo"], c["hi"]) for _ in range(c["R"] - 1)]


def _news(c):
    """New tokens of each request: one each, or up to twice `new`, the first the most."""
    r = random.Random("new %(R)d %(new)d" % c)
    return [c["new"]] * c["R"] if c["new"] == 1 else [2 * c["new"]] + [r.randint(0, 2 * c["new"]) for _ in range(c["R"] - 1)]


def _befores(c):
    """Tokens that the append's requests already have."""
    r = random.Random("before %(R)d %(P)d" % c)
    return [r.randint(0, 3 * c["P"]) for _ in range(c["R"])]


def _drops(c):
    """Tokens that come off the end of each request."""
    r = random.Random("drop %(R)d %(drop)d" % c)
    return [r.randint(0, c["drop"]) for _ in range(c["R"])]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _quantised(g, n):
    """Bytes of two E2M1 codes and E4M3 scales as blocks of 16 normally distributed values give them."""
    x = torch.randn(n, 16, generator=g, device=DEV)
    scale = (x.abs().amax(1, keepdim=True) / 6).to(torch.float8_e4m3fn)
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    code = torch.bucketize(x.abs() / scale.float(), borders) + 8 * (x < 0)
    code = code.view(-1, 2)
    return (code[:, 0] + 16 * code[:, 1]).to(torch.uint8), scale.view(-1).view(torch.uint8)


def _picks(g, of, shape):
    """A tensor of values picked out of `of`, in pieces."""
    out = torch.empty(shape, dtype=torch.uint8, device=DEV)
    flat, step = out.view(-1), 1 << 28
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        flat[i:i + n] = of[torch.randint(0, of.numel(), (n,), generator=g, device=DEV, dtype=torch.int32)]
    return out


def _pool(g, pages, c):
    """Codes [pages, heads, tokens, D / 2], whichever of heads and tokens lies further out in memory, and scales."""
    codes, scales = _quantised(g, 1 << 15)
    shape = (pages, c["Hkv"], c["P"]) if c["layout"] == "heads" else (pages, c["P"], c["Hkv"])
    codes = _picks(g, codes, (*shape, c["D"] // 2))
    codes = codes if c["layout"] == "heads" else codes.transpose(1, 2)
    return codes, _picks(g, scales, (pages, c["Hkv"], c["P"], c["D"] // 16))


def _exponents(g, heads):
    return torch.randint(-2, 2, (heads,), generator=g, device=DEV, dtype=torch.int32)


def _table(g, lens, P, spare):
    """A table of pages in random order; entries past a request's length hold any page."""
    need = torch.tensor([-(-n // P) for n in lens], device=DEV)
    W, total = max(1, int(need.max())), int(need.sum())
    pages = total + spare
    perm = torch.randperm(pages, generator=g, device=DEV)
    col = torch.arange(W, device=DEV)
    at = (need.cumsum(0) - need)[:, None] + col
    return torch.where(col < need[:, None], perm[at.clamp(max=pages - 1)], perm[0]).int(), pages


def _frequencies(c):
    """[axes, rot / 2]: a pair turns with one axis (the pairs dealt out to the axes in turn), at 10000^(-2j/rot) radians a position."""
    j = torch.arange(c["rot"] // 2, device=DEV)
    f = torch.exp(j * (-2 / c["rot"] * math.log(10000.0)))
    return torch.where(j % c["axes"] == torch.arange(c["axes"], device=DEV)[:, None], f, 0.0).float()


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "rope":
        T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
        fused = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device=DEV).bfloat16()  # queries, keys and values of a layer
        s["q"], s["k"] = fused[:, :Hq * D].view(T, Hq, D), fused[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
        s["positions"] = torch.randint(0, c["far"], (c["axes"], T), generator=g, device=DEV, dtype=torch.int32)
        s["freqs"] = _frequencies(c)
        for n in ("q_weight", "k_weight"):
            s[n] = (1 + 0.2 * torch.randn(D, generator=g, device=DEV)).bfloat16() if c["norm"] else None
        return s
    if c["op"] == "verify":
        # Drafts come from the draft model's distributions, which are near the target's; without
        # these they come from the target's (a lookup of earlier text gives likely tokens).
        R, G, V = c["R"], c["G"], c["V"]
        logits = torch.randn(R, G, V, generator=g, device=DEV) * 2.5
        s["target"] = torch.softmax(logits, -1)
        near = torch.softmax(logits[:, :G - 1] + 0.5 * torch.randn(R, G - 1, V, generator=g, device=DEV), -1)
        s["draft"] = near if c["given"] and G > 1 else None
        u = torch.rand(R, G - 1, 1, generator=g, device=DEV)
        s["tokens"] = torch.searchsorted(near.cumsum(-1), u).clamp(max=V - 1).squeeze(-1).int()
        s["accept"], s["sample"] = torch.rand(R, G - 1, generator=g, device=DEV), torch.rand(R, generator=g, device=DEV)
        return s
    if c["op"] == "trim":
        lens = _lengths(c)
        table, pages = _table(g, lens, c["P"], 64)
        used = torch.zeros(pages, dtype=torch.bool, device=DEV)
        col = torch.arange(table.shape[1], device=DEV)
        used[table[col < torch.tensor([-(-n // c["P"]) for n in lens], device=DEV)[:, None]].long()] = True
        free = torch.nonzero(~used).view(-1).int()
        taken = int(torch.randint(0, pages, (1,), generator=g, device=DEV))
        s["ring"] = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
        s["ring"][(taken + torch.arange(len(free), device=DEV)) % pages] = free
        s |= {"lengths": _i32(lens), "drop": _i32(_drops(c)), "table": table, "state": torch.tensor([taken, taken + len(free)], dtype=torch.int64, device=DEV)}
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
        fused = (fused * torch.exp2(torch.randint(-3, 4, (T, 1), generator=g, device=DEV).float())).bfloat16()
        s["k"] = fused[:, Hkv * D:2 * Hkv * D].view(T, Hkv, D)
        s["v"] = fused[:, 2 * Hkv * D:].view(T, Hkv, D)
        b = torch.randn(pages, Hkv, 2, D, generator=g, device=DEV)
        s["bounds"] = torch.stack([b.amax(2), b.amin(2)], 2).bfloat16()
    else:
        lens = _lengths(c)
        table, pages = _table(g, lens, P, 5)
        s |= {"table": table, "lengths": _i32(lens), "q": torch.randn(c["R"] * c["G"], c["Hq"], D, generator=g, device=DEV).bfloat16()}
        if c["K"]:
            # As the select leaves them: ascending, with -1 past a row's count.
            B, W, K = c["R"] * c["G"], table.shape[1], c["K"]
            have = torch.tensor([-(-n // P) for n in lens], device=DEV).repeat_interleave(c["G"])[:, None, None]
            score = torch.rand(B, Hkv, W, generator=g, device=DEV).masked_fill(torch.arange(W, device=DEV) >= have, -1.0)
            top = score.topk(min(K, W), -1).indices
            lists = torch.where(top < have, top, W).sort(-1).values
            s["counts"] = (lists < W).sum(-1).int()
            s["lists"] = torch.where(lists < W, lists, -1).int().contiguous()
    for n in "kv":
        s[n + "_pool"], s[n + "_scales"] = _pool(g, pages, c)
        s[n + "_exp"] = _exponents(g, Hkv)
    return s


# ---- one pass ---------------------------------------------------------------------------------------------------

def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _own_rope(s):
    from sparse_mla_decode_gb300 import binding
    if "out" not in s:
        s["out"] = {n + "_out": torch.empty(s[n].shape, dtype=torch.bfloat16, device=DEV) for n in "qk"}
    q, k = binding.qk_norm_rope(s["q"], s["k"], s["positions"], s["freqs"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                                interleaved=s["case"]["inter"], **s["out"])
    return {"q": q, "k": k}


def _cache(s):
    from sparse_mla_decode_gb300 import binding
    if "cache" not in s:
        s["cache"] = binding.PagedCache4(s["k_pool"], s["v_pool"], s["k_scales"], s["v_scales"], s["k_exp"], s["v_exp"], s.get("bounds"))
    return s["cache"]


def _own_append(s):
    from sparse_mla_decode_gb300 import binding
    if "out" not in s:
        s["out"] = {n: torch.empty(s["slots"].numel(), s["case"]["Hkv"], s["case"]["D"], dtype=torch.bfloat16, device=DEV) for n in "kv"}
    binding.paged4_append(_cache(s), s["k"], s["v"], s["slots"])
    k, v = binding.paged4_read(_cache(s), s["slots"], **s["out"])
    return {"k": k, "v": v, "bounds": s["bounds"]}


def _own_decode(s):
    from sparse_mla_decode_gb300 import binding
    c, q = s["case"], s["q"]
    if "out" not in s:
        s["out"], s["lse"] = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float32, device=DEV)
        s["workspace"] = torch.zeros(binding.paged4_workspace_bytes(_cache(s)), dtype=torch.uint8, device=DEV)
    out, lse = binding.paged4_decode(q, _cache(s), s["table"], s["lengths"], c["D"] ** -0.5, row_group=c["G"], block_lists=s.get("lists"),
                                     block_counts=s.get("counts"), out=s["out"], lse=s["lse"], workspace=s["workspace"])
    return {"out": out, "lse": lse}


def _own_verify(s):
    from sparse_mla_decode_gb300 import binding
    c = s["case"]
    if "out" not in s:
        s["out"] = {"out_tokens": torch.empty(c["R"], c["G"], dtype=torch.int32, device=DEV),
                    **{n: torch.empty(c["R"], dtype=torch.int32, device=DEV) for n in ("accepted", "rejected")}}
    tokens, accepted, rejected = binding.verify_drafts(s["target"], s["tokens"], s["accept"], s["sample"], draft=s["draft"], **s["out"])
    return {"tokens": tokens, "accepted": accepted, "rejected": rejected}


def _own_trim(s):
    from sparse_mla_decode_gb300 import binding
    if "out" not in s:
        s["out"] = {"new_lengths": torch.empty_like(s["lengths"]), "new_state": torch.empty_like(s["state"])}
    lengths, state = binding.block_trim(s["lengths"], s["drop"], s["table"], s["ring"], s["state"], s["case"]["P"], **s["out"])
    return {"lengths": lengths, "state": state, "ring": s["ring"]}


_own = {"rope": _own_rope, "append": _own_append, "decode": _own_decode, "verify": _own_verify, "trim": _own_trim}


def _turned(x, weight, cos, sin, inter):
    """One side of a layer's heads [T, H, D]: norm and rotation; cos and sin [T, 1, rot / 2]."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
    half = cos.shape[-1]
    turn, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (turn[..., 0::2], turn[..., 1::2]) if inter else (turn[..., :half], turn[..., half:])
    c, d = a * cos - b * sin, a * sin + b * cos
    turn = torch.stack([c, d], -1).flatten(-2) if inter else torch.cat([c, d], -1)
    return torch.cat([turn, rest], -1).bfloat16()


def _plain_rope(s):
    angle = torch.matmul(s["positions"].double().t(), s["freqs"].double())[:, None]
    cos, sin = angle.cos().float(), angle.sin().float()
    return {n: _turned(s[n], s[n + "_weight"], cos, sin, s["case"]["inter"]) for n in "qk"}


def _powers(e):
    """2^e in 32 bits, exactly (|e| <= 100)."""
    return ((e + 127) << 23).int().view(torch.float32)


def _encode(x, exp):
    """Codes, two a byte, and scales of x [T, heads, D]."""
    x = (x.float() * _powers(-exp)[:, None]).unflatten(-1, (-1, 16))
    scale = (x.abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn)
    y = x / torch.where(scale.float() > 0, scale.float(), 1.0)[..., None]
    y = torch.where(scale.float()[..., None] > 0, y, 0.0)
    a = y.abs()
    code = (a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)  # ties to even codes
    code = (code + 8 * (y < 0)).flatten(-2)
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), scale.view(torch.uint8)


def _decode(codes, scales, exp):
    """Values of codes [.., D / 2] and scales [.., D / 16]; exp: exponents that broadcast over [..]."""
    table = torch.tensor([*MAGNITUDES, *(-m for m in MAGNITUDES)], device=DEV)
    x = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).flatten(-2)
    return (x.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2) * _powers(exp)[..., None]


def _over_pages(start, at, x, how):
    """The extremes of x's rows over the rows of each page, from `start` on."""
    return start.scatter_reduce(0, at.view(-1, *[1] * (x.dim() - 1)).expand_as(x), x, how)


def _stored(s, n, page, offset):
    """Keys or values written into their slots, then read back."""
    codes, scales = s[n + "_pool"], s[n + "_scales"]
    codes[page, :, offset], scales[page, :, offset] = _encode(s[n], s[n + "_exp"])
    return _decode(codes[page, :, offset], scales[page, :, offset], s[n + "_exp"]).bfloat16()


def _plain_append(s):
    P, slots = s["case"]["P"], s["slots"].long()
    page, offset = slots // P, slots % P
    got = {n: _stored(s, n, page, offset) for n in "kv"}
    touched, at = torch.unique(page, return_inverse=True)
    first = torch.full((touched.numel(),), P, device=DEV).scatter_reduce(0, at, offset, "amin")
    k = s["k"].float()
    inf = torch.full((touched.numel(), *k.shape[1:]), math.inf, device=DEV)
    was = s["bounds"][touched].float()
    part = (first > 0)[:, None, None]
    hi = _over_pages(torch.where(part, was[:, :, 0], -inf), at, k, "amax")
    lo = _over_pages(torch.where(part, was[:, :, 1], inf), at, k, "amin")
    s["bounds"][touched] = torch.stack([hi, lo], 2).bfloat16()
    return {**got, "bounds": s["bounds"]}


def _limits(s):
    """The tokens that each row sees: verify row i of G sees the first length - G + 1 + i."""
    G = s["case"]["G"]
    return (s["lengths"].long()[:, None] - G + 1 + torch.arange(G, device=DEV)).clamp(min=0)


def _softmax_of(logits, v):
    """Rows of logits (masked: -inf) over values: the output and the natural logarithm of the sum; nothing seen: 0 and -inf."""
    m = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - m.masked_fill(m == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / total.masked_fill(total == 0, 1.0)
    return out, (m + torch.log(total)).squeeze(-1)


def _plain_decode(s):
    c = s["case"]
    R, G, Hkv, g, P, D = c["R"], c["G"], c["Hkv"], c["Hq"] // c["Hkv"], c["P"], c["D"]
    q, table, lim = s["q"].float() * D ** -0.5, s["table"].long(), _limits(s)
    if c["K"]:
        lists = s["lists"].long()
        listed_ = torch.arange(lists.shape[-1], device=DEV) < s["counts"][:, :, None]
        pages = table.repeat_interleave(G, 0)[:, None].expand(-1, Hkv, -1).gather(2, lists.clamp(min=0))  # [B, Hkv, K]
        heads = torch.arange(Hkv, device=DEV)[None, :, None]
        seen = ((lists[..., None] * P + torch.arange(P, device=DEV) < lim.view(-1)[:, None, None, None]) & listed_[..., None]).flatten(2)[:, :, None]
        values = lambda n: _decode(s[n + "_pool"][pages, heads], s[n + "_scales"][pages, heads], s[n + "_exp"][:, None, None]).flatten(2, 3)  # noqa: E731
        logits = torch.matmul(q.view(-1, Hkv, g, D), values("k").transpose(-1, -2)).masked_fill(~seen, -math.inf)
        out, lse = _softmax_of(logits, values("v"))
    else:
        values = lambda n: _decode(s[n + "_pool"][table], s[n + "_scales"][table], s[n + "_exp"][:, None]).transpose(1, 2).flatten(2, 3)  # noqa: E731  [R, Hkv, W * P, D]
        rows = q.view(R, G, Hkv, g, D).transpose(1, 2).flatten(2, 3)
        at = torch.arange(table.shape[1] * P, device=DEV)
        seen = (at < lim[:, :, None]).repeat_interleave(g, 1)[:, None]  # [R, 1, G * g, W * P]
        logits = torch.matmul(rows, values("k").transpose(-1, -2)).masked_fill_(~seen, -math.inf)
        out, lse = _softmax_of(logits, values("v"))
        out, lse = (x.view(R, Hkv, G, g, *x.shape[3:]).transpose(1, 2).flatten(0, 1) for x in (out, lse))
    return {"out": out.reshape(R * G, c["Hq"], D).bfloat16(), "lse": lse.reshape(R * G, c["Hq"])}


def _share(p):
    """Probabilities as whole multiples of 2^-40: sums of them do not depend on their order."""
    return (p.clamp(0, 1) * 2.0 ** 40).floor().long()


def _plain_verify(s):
    p, q, tokens = s["target"], s["draft"], s["tokens"].long()
    R, G, V = p.shape
    row = torch.arange(R, device=DEV)
    drafted = (tokens >= 0) & (tokens < V)
    at = tokens.clamp(0, V - 1)[..., None]
    pd = p[:, :G - 1].gather(-1, at).squeeze(-1).double()
    qd = q.gather(-1, at).squeeze(-1).double() if q is not None else torch.ones_like(pd)
    good = drafted & (s["accept"].double() * qd < pd)
    accepted = good.int().cumprod(1).sum(1)
    last = _rejected(drafted, accepted)  # whether a draft was rejected there
    left = p[row, accepted]
    if q is not None:
        left = left - torch.where(last[:, None], q[row, accepted.clamp(max=G - 2)], 0.0)
    elif G > 1:
        gone = tokens.gather(1, accepted.clamp(max=G - 2)[:, None]).clamp(0, V - 1)
        left = left.scatter_add(1, gone, -last[:, None].float())
    w = _share(left)
    w = torch.where(w.sum(1, keepdim=True) > 0, w, _share(p[row, accepted]))
    total = w.sum(1)
    u = (s["sample"].double() * 2.0 ** 31).floor().long().clamp(0, (1 << 31) - 1)
    t = u * (total >> 32) * 2 + ((u * (total & 0xffffffff)) >> 31)  # floor(u * total / 2^31)
    drawn = (w.cumsum(1) <= t[:, None]).sum(1)
    col = torch.arange(G, device=DEV)
    out = torch.where(col < accepted[:, None], torch.cat([tokens, tokens.new_zeros(R, 1)], 1), -1)
    out = torch.where(col == accepted[:, None], drawn[:, None], out)
    return {"tokens": out.int(), "accepted": accepted.int(), "rejected": (G - 1 - accepted).int()}


def _rejected(drafted, at):
    """drafted[r, at[r]], false past its end."""
    return torch.cat([drafted, torch.zeros_like(at, dtype=torch.bool)[:, None]], 1).gather(1, at[:, None].long()).squeeze(1)


def _before(x):
    return x.cumsum(0) - x


def _plain_trim(s):
    P, table, ring = s["case"]["P"], s["table"], s["ring"]
    length = s["lengths"].long()
    new = (length - s["drop"].long().clamp(min=0)).clamp(min=0)
    have, keep = (length + P - 1) // P, (new + P - 1) // P
    col = torch.arange(table.shape[1], device=DEV)
    at = s["state"][1] + _before(have - keep)[:, None] + col - keep[:, None]
    goes = (col >= keep[:, None]) & (col < have[:, None])
    pages = ring.numel()
    put = torch.where(goes, at % pages, pages)
    s["ring"] = torch.cat([ring, ring.new_zeros(1)]).scatter(0, put.view(-1), table.reshape(-1))[:pages]
    return {"lengths": new.int(), "state": torch.stack([s["state"][0], s["state"][1] + (have - keep).sum()]), "ring": s["ring"]}


_plain = {"rope": _plain_rope, "append": _plain_append, "decode": _plain_decode, "verify": _plain_verify, "trim": _plain_trim}


# ---- what a pass cannot do without ----------------------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "rope":
        values = c["T"] * (c["Hq"] + c["Hkv"]) * c["D"]
        return {"bytes": 4 * values + 4 * c["T"] * c["axes"] + 2 * c["axes"] * c["rot"], "flops": 6.0 * values}
    if c["op"] == "verify":  # one row of each request, and its draft's
        return {"bytes": c["R"] * (c["V"] * (8 if c["given"] and c["G"] > 1 else 4) + 20 * c["G"]), "flops": 2.0 * c["R"] * c["V"]}
    P = c["P"]
    up = lambda n: -(-max(0, n) // P)  # noqa: E731
    if c["op"] == "trim":
        back = sum(up(n) - up(n - d) for n, d in zip(_lengths(c), _drops(c)))
        return {"bytes": 12 * c["R"] + 32 + 8 * back, "flops": 0}
    D, Hkv = c["D"], c["Hkv"]
    token = D + D // 8  # bytes of a token's keys and values, one head
    if c["op"] == "append":  # written, and read back
        new = _news(c)
        pages = sum(up(a + n) - a // P for a, n in zip(_befores(c), new) if n)
        return {"bytes": sum(new) * (8 + Hkv * (8 * D + 2 * token)) + pages * Hkv * 4 * D, "flops": 0}
    lens, G, Hq = _lengths(c), c["G"], c["Hq"]
    io = c["R"] * G * Hq * (4 * D + 4)
    if c["K"]:
        tokens = sum(min(max(0, n - G + 1 + i), c["K"] * P) for n in lens for i in range(G))  # of each row and kv head
        return {"bytes": io + tokens * Hkv * token + -(-tokens // P) * Hkv * 8, "flops": 4.0 * tokens * Hq * D}
    return {"bytes": io + sum(lens) * Hkv * token + sum(map(up, lens)) * 4,
            "flops": 4.0 * D * Hq * sum(max(0, n - G + 1 + i) for n in lens for i in range(G))}


# ---- 64 bits --------------------------------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] in ("verify", "trim"):
        return None  # whole numbers
    return {"rope": _exact_rope, "append": _exact_append, "decode": _exact_decode}[case["op"]](prepare(case, seed))


def _exact_rope(s):
    c, out = s["case"], {}
    angle = sum(s["positions"][a].double()[:, None] * s["freqs"][a].double() for a in range(c["axes"]))
    turn = torch.polar(torch.ones_like(angle), angle)  # [T, rot / 2]
    n = c["rot"] // 2
    first = torch.arange(n, device=DEV) * (2 if c["inter"] else 1)
    second = first + (1 if c["inter"] else n)
    for name in "qk":
        y = s[name].double()
        if s[name + "_weight"] is not None:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / c["D"] + EPS) * s[name + "_weight"].double()
        z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
        y = y.clone()
        y[..., first], y[..., second] = z.real, z.imag
        out[name] = y
    return out


def _e4m3_values():
    """The 256 values of E4M3 from its definition: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN."""
    v = []
    for b in range(128):
        e, m = b >> 3, b & 7
        v.append(math.nan if b == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return torch.tensor(v + [-x for x in v], dtype=torch.float64, device=DEV)


def _e2m1_values():
    """The 16 values of E2M1 from its definition: sign, 2 exponent bits (bias 1), 1 mantissa bit."""
    v = [(b & 1) * 0.5 if b < 2 else (2 + (b & 1)) * 2.0 ** ((b >> 1) - 2) for b in range(8)]
    return torch.tensor(v + [-x for x in v], dtype=torch.float64, device=DEV)


def _nearest(x, v):
    """The value of v (ascending, of codes 0, 1, ..) nearest to |x|, with x's sign; ties to the even code, what is larger to the largest."""
    a = x.abs()
    below = (torch.searchsorted(v, a.contiguous(), right=True) - 1).clamp(0, v.numel() - 1)
    above = (below + 1).clamp(max=v.numel() - 1)
    d, u = a - v[below], v[above] - a
    near = torch.where((u < d) | ((u == d) & (above % 2 == 0)), above, below)
    return torch.copysign(v[near], x)


def _exact_append(s):
    P, got = s["case"]["P"], {}
    for n in "kv":
        x = s[n].double() * torch.pow(2.0, -s[n + "_exp"].double())[:, None]
        x = x.view(*x.shape[:2], -1, 16)
        scale = _nearest(x.abs().amax(-1, keepdim=True) / 6, _e4m3_values()[:127])
        y = _nearest(x / scale.clamp(min=2.0 ** -20), _e2m1_values()[:8]) * scale
        got[n] = y.flatten(2) * torch.pow(2.0, s[n + "_exp"].double())[:, None]
    slots, b, k = s["slots"].tolist(), s["bounds"].double(), s["k"].double()
    i = 0
    for j in range(1, len(slots) + 1):
        if j == len(slots) or slots[j] // P != slots[i] // P:
            p = slots[i] // P
            y = k[i:j] if slots[i] % P == 0 else torch.cat([k[i:j], b[p].transpose(0, 1)])
            b[p] = torch.stack([y.amax(0), y.amin(0)], 1)
            i = j
    return {**got, "bounds": b}


def _exact_decode(s):
    c, v4, v8 = s["case"], _e2m1_values(), _e4m3_values()
    G, Hkv, g, P, D = c["G"], c["Hkv"], c["Hq"] // c["Hkv"], c["P"], c["D"]
    out = torch.zeros(c["R"] * G, Hkv, g, D, dtype=torch.float64, device=DEV)
    lse = torch.full((c["R"] * G, Hkv, g), -math.inf, dtype=torch.float64, device=DEV)
    heads = torch.arange(Hkv, device=DEV)[:, None]

    def values(n, pages):
        codes = s[n + "_pool"][pages, heads].long()  # [Hkv, blocks, P, D / 2]
        x = torch.empty(*codes.shape[:-1], D, dtype=torch.float64, device=DEV)
        x[..., 0::2], x[..., 1::2] = v4[codes % 16], v4[codes // 16]
        x = x * v8[s[n + "_scales"][pages, heads].long()].repeat_interleave(16, -1)
        return x.flatten(1, 2) * torch.pow(2.0, s[n + "_exp"].double())[:, None, None]

    for r, n in enumerate(s["lengths"].tolist()):
        for i in range(G if n else 0):
            b, lim = r * G + i, max(0, n - G + 1 + i)
            if not lim:
                continue
            blocks = s["lists"][b].long().clamp(min=0) if c["K"] else torch.arange(-(-n // P), device=DEV).expand(Hkv, -1)
            pages = s["table"][r].long()[blocks]  # [Hkv, blocks]
            pos = (blocks[..., None] * P + torch.arange(P, device=DEV)).flatten(1)
            seen = pos < lim
            if c["K"]:
                seen = seen & (torch.arange(blocks.shape[1], device=DEV) < s["counts"][b][:, None]).repeat_interleave(P, 1)
            q = s["q"][b].double().view(Hkv, g, D)
            x = torch.einsum("hgd,hnd->hgn", q, values("k", pages)) / math.sqrt(D)
            x = x.masked_fill(~seen[:, None], -math.inf)
            lse[b] = torch.logsumexp(x, -1)
            out[b] = torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1), values("v", pages))
    return {"out": out.view(c["R"] * G, c["Hq"], D), "lse": lse.view(c["R"] * G, c["Hq"])}
