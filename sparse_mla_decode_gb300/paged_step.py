"""Decode steps over a paged cache, put together from the library's calls.

    python -m sparse_mla_decode_gb300.paged_step [--requests 32] [--context 32768]
        [--steps 8] [--pages 64] [--bits 8] [--drafts 0]

Requests of up to ``--context`` tokens hold pages of a grouped-query cache (64
query heads over 8 key/value heads of 128 columns). A prompt is written once;
then every step gives each request a slot for its new token (block_tables),
writes the token's keys and values (paged_append), scores the pages for the
step's queries (block_scores), selects ``--pages`` of them for each request and
key/value head (topk_select, the first and the last two always among them)
and attends over those (paged_decode). ``--bits 4``: the cache is in E2M1 with block scales
(paged4_append, paged4_decode), after the norm of queries and keys and the position
rotation (qk_norm_rope). ``--drafts N``: a step writes and attends N drafted tokens more
for each request, their verification against random distributions (verify_drafts) follows, and what
is refused gives its pages back (block_trim). Values are random. The step is
captured in a CUDA graph and replayed; the same step with attention over all
tokens is timed beside it, and the selected pages' share of the attention
weight is printed.
"""
from __future__ import annotations

import argparse
import math


class PagedStep:
    """The buffers of a batch of requests and their decode step. ``pages`` None:
    attention over all tokens."""

    def __init__(self, requests, width, pool_pages, q_heads=64, heads=8, head_dim=128, page_size=64,
                 pages=None, device="cuda", bits=8):
        import torch
        from . import binding

        kind = {8: binding.PagedCache, 4: binding.PagedCache4}[bits]
        self.cache, self.bits = kind.empty(pool_pages, heads, page_size, head_dim, device=device), bits
        self.pages, self.sm_scale = pages, head_dim ** -0.5
        self.table = torch.zeros((requests, width), dtype=torch.int32, device=device)
        self.ring = torch.arange(pool_pages, dtype=torch.int32, device=device)
        # Lengths and pool state, of this step and of the next: block_tables writes from one
        # to the other.
        self.lengths = [torch.zeros(requests, dtype=torch.int32, device=device) for _ in range(2)]
        self.state = [torch.tensor([0, pool_pages], dtype=torch.int64, device=device) for _ in range(2)]
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        room = binding.paged_workspace_bytes if bits == 8 else binding.paged4_workspace_bytes
        self.workspace = torch.zeros(room(self.cache), dtype=torch.uint8, device=device)
        self.now = 0

    def grant(self, new_tokens, max_tokens):
        """Slots and positions of new_tokens [R] int32 more tokens (below 0: a
        request has ended). Returns (starts, slots, positions)."""
        from . import binding

        a, b = self.now, 1 - self.now
        _, _, starts, slots, positions = binding.block_tables(
            self.lengths[a], new_tokens, self.table, self.ring, self.state[a], self.cache.page_size,
            max_tokens, new_lengths=self.lengths[b], new_state=self.state[b], status=self.status)
        self.now = b
        return starts, slots, positions

    def write(self, k, v, slots):
        """Keys and values [T, heads, head_dim] bf16 of granted tokens."""
        from . import binding

        (binding.paged_append if self.bits == 8 else binding.paged4_append)(self.cache, k, v, slots)

    def attend(self, q, row_group=1):
        """Attention of the queries [R * row_group, q_heads, head_dim] bf16. Returns
        (out, lse)."""
        from . import binding

        lengths = self.lengths[self.now]
        lists = counts = None
        if self.pages is not None:
            scores = binding.block_scores(q, self.cache, self.table, lengths, row_group=row_group,
                                          keep_first=1, keep_last=2)
            B, heads, width = scores.shape
            # Rows of the scores lie a multiple of 8 apart; the select reads `width` of each.
            flat = scores.as_strided((B * heads, width), (scores.stride(1), 1))
            idx, cnt = binding.topk_select(flat, self.pages)
            lists, counts = idx.view(B, heads, self.pages), cnt
        decode = binding.paged_decode if self.bits == 8 else binding.paged4_decode
        return decode(q, self.cache, self.table, lengths, self.sm_scale, row_group=row_group,
                      block_lists=lists, block_counts=counts, status=self.status,
                      workspace=self.workspace)

    def keep(self, target, tokens, accept, sample, draft=None):
        """Verification of the last G - 1 tokens that each request was granted (verify_drafts' arguments);
        those that are refused come off, and their pages go back. A request that the last grant gave n < G tokens
        has n - 1 drafts (tokens outside the vocabulary behind them); one that it gave none (idle, refused or
        ended) keeps what it holds, and its results mean nothing. Returns (out_tokens, accepted)."""
        from . import binding

        a, b = self.now, 1 - self.now
        out, accepted, rejected = binding.verify_drafts(target, tokens, accept, sample, draft=draft)
        # `rejected` counts G - 1 drafts for every request. Those that a request was not granted (its length
        # grew by less than G over the grant) hold no slots; a drop below 0 takes nothing.
        rejected += (self.lengths[a] - self.lengths[b]).sub_(target.shape[1]).clamp_(max=0)
        binding.block_trim(self.lengths[a], rejected, self.table, self.ring, self.state[a],
                           self.cache.page_size, new_lengths=self.lengths[b], new_state=self.state[b])
        self.now = b
        return out, accepted


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=32)
    ap.add_argument("--context", type=int, default=32768)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--pages", type=int, default=64)
    ap.add_argument("--bits", type=int, default=8, choices=(8, 4))
    ap.add_argument("--drafts", type=int, default=0)
    args = ap.parse_args(argv)
    if not 0 <= args.drafts <= 7:
        ap.error("--drafts must be 0 to 7")
    for name in ("requests", "context", "steps", "pages"):
        if getattr(args, name) < 1:
            ap.error(f"--{name} must be at least 1")
    if args.requests > 8192:
        ap.error("--requests must be at most 8192")
    replays = (args.steps + 1) // 2  # of two steps each

    import torch
    from . import binding

    R, P, heads, q_heads, D = args.requests, 64, 8, 64, 128
    g = torch.Generator(device="cuda").manual_seed(0)
    lengths = torch.randint(max(1, args.context // 4), args.context + 1, (R,), generator=g, device="cuda")
    G = 1 + args.drafts
    width = -(-(args.context + G * (4 * args.steps + 8)) // P)
    s = PagedStep(R, width, R * width, q_heads, heads, D, P, pages=args.pages, bits=args.bits)

    def random(n, h):
        return torch.randn(n, h, D, generator=g, device="cuda").bfloat16()

    freqs = torch.exp(torch.arange(D // 2, device="cuda") * (-2 / D * math.log(10000.0)))
    weight = torch.ones(D, dtype=torch.bfloat16, device="cuda")

    def turn(q, k, positions):
        """What is asked with and written: as given in 8 bits, normed and rotated in 4."""
        if args.bits == 8:
            return q, k
        return binding.qk_norm_rope(q, k, positions, freqs, weight, weight)

    # The prompts, in pieces as a scheduler would admit them.
    left, T = lengths.clone(), 65536
    while int(left.sum()):
        share = torch.minimum(left, torch.tensor(T // R, device="cuda"))
        starts, slots, positions = s.grant(share.int(), T)
        n = int(starts[-1])
        k, _ = turn(random(n, heads), None, positions[:n])
        s.write(k, random(n, heads), slots[:n].contiguous())
        left -= share
    assert int(s.status) == 0, "a request was refused"

    new = torch.full((R,), G, dtype=torch.int32, device="cuda")
    q, k, v = random(R * G, q_heads), random(R * G, heads), random(R * G, heads)
    if G > 1:
        V = 32768
        target = torch.softmax(2 * torch.randn(R, G, V, generator=g, device="cuda"), -1)
        tokens = target[:, 1:].argmax(-1).int()
        accept = 0.1 * torch.rand(R, G - 1, generator=g, device="cuda")
        sample = torch.rand(R, generator=g, device="cuda")

    def step():
        _, slots, positions = s.grant(new, R * G)
        qt, kt = turn(q, k, positions)
        s.write(kt, v, slots)
        out = s.attend(qt, row_group=G)
        if G > 1:
            s.keep(target, tokens, accept, sample)
        return out

    times = {}
    for name, pages in (("selected", args.pages), ("all", None)):
        s.pages = pages
        step(), step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):  # two steps: the buffers of lengths and state alternate
            step()
            result = step()
        graph.replay()
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for _ in range(replays):
            graph.replay()
        end.record()
        torch.cuda.synchronize()
        times[name] = start.elapsed_time(end) * 1e3 / (2 * replays)
        assert int(s.status) == 0, "device status"
        if pages is not None:
            last = s.lengths[s.now][:, None] - G + torch.arange(G, dtype=torch.int32, device="cuda")
            qt, _ = turn(q, None, last.flatten())  # the queries of the last G tokens
            _, lse = s.attend(qt, row_group=G)
            s.pages = None
            _, lse_all = s.attend(qt, row_group=G)
            kept = torch.exp(lse - lse_all)[lse_all > -math.inf].mean()  # of rows that see a token
        del result
    n = int(s.lengths[s.now].sum())
    print(f"{R} requests, {n} tokens ({n * heads * D * (2 if args.bits == 8 else 1.125) / 1e9:.2f} GB of keys and "
          "values)")
    print(f"step over {args.pages} pages of each request and head: {times['selected']:.1f} us "
          f"({100 * float(kept):.1f}% of the attention weight of random values)")
    print(f"step over all tokens: {times['all']:.1f} us")
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
