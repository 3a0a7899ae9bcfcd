"""Decode steps over a paged cache, put together from the library's calls.

    python -m sparse_mla_decode_gb300.paged_step [--requests 32] [--context 32768]
        [--steps 8] [--pages 64]

Requests of up to ``--context`` tokens hold pages of a grouped-query cache (64
query heads over 8 key/value heads of 128 columns). A prompt is written once;
then every step gives each request a slot for its new token (block_tables),
writes the token's keys and values (paged_append), scores the pages for the
step's queries (block_scores), selects ``--pages`` of them for each request and
key/value head (topk_select, the first and the last two always among them)
and attends over those (paged_decode). Values are random. The step is
captured in a CUDA graph and replayed; the same step with attention over all
tokens is timed beside it, and the selected pages' share of the attention
weight is printed.
"""
from __future__ import annotations

import argparse


class PagedStep:
    """The buffers of a batch of requests and their decode step. ``pages`` None:
    attention over all tokens."""

    def __init__(self, requests, width, pool_pages, q_heads=64, heads=8, head_dim=128, page_size=64,
                 pages=None, device="cuda"):
        import torch
        from . import binding

        self.cache = binding.PagedCache.empty(pool_pages, heads, page_size, head_dim, device=device)
        self.pages, self.sm_scale = pages, head_dim ** -0.5
        self.table = torch.zeros((requests, width), dtype=torch.int32, device=device)
        self.ring = torch.arange(pool_pages, dtype=torch.int32, device=device)
        # Lengths and pool state, of this step and of the next: block_tables writes from one
        # to the other.
        self.lengths = [torch.zeros(requests, dtype=torch.int32, device=device) for _ in range(2)]
        self.state = [torch.tensor([0, pool_pages], dtype=torch.int64, device=device) for _ in range(2)]
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.workspace = torch.zeros(binding.paged_workspace_bytes(self.cache), dtype=torch.uint8,
                                     device=device)
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

        binding.paged_append(self.cache, k, v, slots)

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
        return binding.paged_decode(q, self.cache, self.table, lengths, self.sm_scale,
                                    row_group=row_group, block_lists=lists, block_counts=counts,
                                    status=self.status, workspace=self.workspace)


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=32)
    ap.add_argument("--context", type=int, default=32768)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--pages", type=int, default=64)
    args = ap.parse_args(argv)
    for name in ("requests", "context", "steps", "pages"):
        if getattr(args, name) < 1:
            ap.error(f"--{name} must be at least 1")
    if args.requests > 8192:
        ap.error("--requests must be at most 8192")
    replays = (args.steps + 1) // 2  # of two steps each

    import torch

    R, P, heads, q_heads, D = args.requests, 64, 8, 64, 128
    g = torch.Generator(device="cuda").manual_seed(0)
    lengths = torch.randint(max(1, args.context // 4), args.context + 1, (R,), generator=g, device="cuda")
    width = -(-(args.context + 4 * args.steps + 8) // P)
    s = PagedStep(R, width, R * width, q_heads, heads, D, P, pages=args.pages)

    def random(n, h):
        return torch.randn(n, h, D, generator=g, device="cuda").bfloat16()

    # The prompts, in pieces as a scheduler would admit them.
    left, T = lengths.clone(), 65536
    while int(left.sum()):
        share = torch.minimum(left, torch.tensor(T // R, device="cuda"))
        starts, slots, _ = s.grant(share.int(), T)
        n = int(starts[-1])
        s.write(random(n, heads), random(n, heads), slots[:n].contiguous())
        left -= share
    assert int(s.status) == 0, "a request was refused"

    one = torch.ones(R, dtype=torch.int32, device="cuda")
    q, k, v = random(R, q_heads), random(R, heads), random(R, heads)

    def step():
        _, slots, _ = s.grant(one, R)
        s.write(k, v, slots)
        return s.attend(q)

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
            _, lse = s.attend(q)
            s.pages = None
            _, lse_all = s.attend(q)
            kept = torch.exp(lse - lse_all).mean()
        del result
    n = int(s.lengths[s.now].sum())
    print(f"{R} requests, {n} tokens ({n * heads * D * 2 / 1e9:.2f} GB of keys and values)")
    print(f"step over {args.pages} pages of each request and head: {times['selected']:.1f} us "
          f"({100 * float(kept):.1f}% of the attention weight of random values)")
    print(f"step over all tokens: {times['all']:.1f} us")
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
