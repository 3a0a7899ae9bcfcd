"""smd_paged4_append in its form for many tokens (a block takes 64 tokens of a head, then the bounds of the runs
that begin among them), on the GPU against the 64-bit oracle, bit for bit. Which form a call takes goes by its
(token, head) pairs; the limit is read where the library has it."""
from __future__ import annotations

import os
import re

import numpy as np
import pytest

from oracle import paged as opaged
from paged4_common import Cache4
from paged_common import bf16, i32
from test_paged4_append_gpu import check, tokens

pytestmark = pytest.mark.gpu
CHUNK = 64


def limit():
    """The most (token, head) pairs that go to the form for few tokens, on this GPU."""
    import torch
    import sparse_mla_decode_gb300 as package
    with open(os.path.join(os.path.dirname(package.__file__), "csrc", "smd_paged4_append.cu")) as f:
        per_sm = re.search(r"constexpr int kFewUnits = (\d+);", f.read())
    return int(per_sm.group(1)) * torch.cuda.get_device_properties(0).multi_processor_count


def spans_of(rng, P, n):
    """(offset, length) of n runs in pages of their own: whole pages, single tokens, short and long pieces."""
    out = []
    for i in range(n):
        o = int(rng.integers(0, P))
        out.append([(0, P), (o, 1), (0, int(rng.integers(1, P + 1))), (o, P - o), (o, min(int(rng.integers(1, 10)), P - o))][i % 5])
    return out


def slots_of(rng, P, need, apart):
    """(slots, pages) of at least `need` live tokens: runs in random pages of their own; `apart`: with slots that
    are skipped between some of them."""
    spans, live = [], 0
    while live < need:
        more = spans_of(rng, P, 50)
        spans += more
        live += sum(n for _, n in more)
    pages = len(spans) + 3
    slots = []
    for page, (o, n) in zip(rng.permutation(pages), spans):
        slots += list(page * P + o + np.arange(n))
        if apart:
            slots += [[], [-1], [pages * P, -7], [2 ** 31 - 1] * 5][rng.integers(0, 4)]
    return np.array(slots), pages


@pytest.mark.parametrize("D,P,heads,layout,fused,exps,apart,bounds", [
    (64, 16, 32, "tokens", 3, True, True, True), (64, 48, 5, "heads", 0, False, False, True),
    (64, 256, 16, "paired", 0, True, True, True), (64, 16, 32, "tokens", 3, True, True, False),
    (128, 64, 16, "heads", 0, True, True, True), (128, 256, 8, "tokens", 1, False, False, True),
    (128, 16, 61, "paired", 0, True, False, True), (128, 64, 16, "heads", 0, True, True, False),
    (256, 80, 16, "heads", 0, True, True, True), (256, 256, 7, "tokens", 2, True, False, True),
    (256, 80, 16, "heads", 0, True, True, False)])
def test_runs_across_chunks(cuda, D, P, heads, layout, fused, exps, apart, bounds):
    rng = np.random.default_rng(D + P + heads + apart)
    slots, pages = slots_of(rng, P, limit() // heads + 1, apart)
    if len(slots) % CHUNK == 0:
        slots = slots[:-1]
    T = len(slots)
    assert T * heads > limit() and T % CHUNK != 0
    check(cuda, Cache4(D + P, pages, heads, P, D, layout, exps), tokens(rng, T, heads, D), slots, fused, bounds)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_request_of_whole_pages_that_begins_inside_a_chunk_and_a_page(cuda, D):
    """Every run but the first begins at another place of its chunk; those of 256 tokens go on over four chunks."""
    rng = np.random.default_rng(D)
    P, heads = 256, 16
    pages = limit() // heads // P + 3
    order = rng.permutation(pages)
    first = 37  # the first page's last tokens
    slots = np.concatenate([order[0] * P + np.arange(P - first, P)] + [p * P + np.arange(P) for p in order[1:]])
    assert len(slots) * heads > limit()
    check(cuda, Cache4(3, pages, heads, P, D), tokens(rng, len(slots), heads, D), slots)


@pytest.mark.parametrize("D,P", [(64, 32), (128, 64), (256, 16)])
@pytest.mark.parametrize("bounds", [True, False])
def test_zeros_nans_infinities_and_extremes(cuda, D, P, bounds):
    rng = np.random.default_rng(D)
    heads = 12
    x = tokens(rng, 32, heads, D)
    for y in x:
        y[0] = 0.0
        y[1, 0] = np.nan
        y[2, 1, 5] = np.nan
        y[3, 2, 7], y[3, 2, 40] = np.inf, -np.inf
        y[4] = opaged.BF16_MAX
        y[5] = -opaged.BF16_MAX
        y[6] = opaged.bf16_round(np.full((heads, D), 2.0 ** -126))
        y[7, 0, :16] = -0.0
        y[8, 1, 16] = np.nan
        y[8, 1, 17] = np.inf
        y[9] = opaged.bf16_round(y[9] * 2.0 ** 60)
        y[10] = opaged.bf16_round(y[10] * 2.0 ** -60)
        y[11:, 7] = np.nan
    n = limit() // heads // 32 + 1
    assert 32 * n * heads > limit()
    order = np.concatenate([rng.permutation(32) for _ in range(n)])  # what meets in a page and a chunk differs
    x = [np.ascontiguousarray(y[order]) for y in x]
    cache = Cache4(7, 32 * n // P + 1, heads, P, D)
    cache.exps = [np.r_[100, -100, 7, -400, 400, rng.integers(-9, 9, heads - 5)], np.r_[-400, 60, 400, rng.integers(-9, 9, heads - 3)]]
    check(cuda, cache, x, np.arange(32 * n), bounds=bounds)


def test_tokens_in_any_order(cuda):
    """Runs of one token, mostly, and slots that are skipped."""
    rng = np.random.default_rng(4)
    D, P, heads = 64, 32, 24
    T = limit() // heads + 1001
    pages = T // P + 40
    slots = rng.permutation(pages * P)[:T]
    slots[rng.random(T) < 0.2] = -1
    slots[rng.random(T) < 0.1] = pages * P + 5
    check(cuda, Cache4(3, pages, heads, P, D), tokens(rng, T, heads, D), slots, bounds=False)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_both_forms_write_the_same(cuda, D):
    """The tokens of one call, and the same in calls below the limit, cut at pages."""
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(D)
    P, heads = 64, 8
    n = limit() // heads // P + 1
    slots = np.concatenate([p * P + np.arange(P) for p in rng.permutation(n)])
    T = len(slots)
    assert T * heads > limit() >= (T - P) * heads
    x = [bf16(y, cuda) for y in tokens(rng, T, heads, D)]
    s = i32(slots, cuda)
    one, parts = (binding.PagedCache4.empty(n, heads, P, D, device=cuda) for _ in "ab")
    binding.paged4_append(one, *x, s)
    for a in range(0, T, 5 * P):
        binding.paged4_append(parts, *(y[a:a + 5 * P] for y in x), s[a:a + 5 * P])
    torch.cuda.synchronize()
    for name in ("k", "v", "k_scales", "v_scales", "bounds"):
        a, b = getattr(one, name), getattr(parts, name)
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name


@pytest.mark.parametrize("D,heads,T", [(64, 11, 5000), (128, 9, 2600), (128, 17, 1300), (128, 17, 2600), (256, 16, 1400), (256, 41, 700)])
def test_heads_that_a_lane_reads_in_several_rounds(cuda, D, heads, T):
    """smd_paged4_read takes 8 heads at a time of those that a unit has; a unit has every `shares`-th head."""
    import torch
    from sparse_mla_decode_gb300 import binding
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    shares = max(1, min(-(-sms * 2 * 128 // (D // 16) // (2 * T)), heads))
    assert -(-heads // shares) > 8
    rng = np.random.default_rng(D + heads)
    cache = Cache4(8, -(-T // 32) + 1, heads, 32, D)
    c = cache.to(cuda)
    slots = rng.permutation(cache.pages * 32)[:T]
    slots[::50] = -1
    got = binding.paged4_read(c, i32(slots, cuda))
    torch.cuda.synchronize()
    for side, t in enumerate(got):
        want = cache.values(side)[slots // 32, :, slots % 32]
        want[::50] = 0
        assert np.array_equal(t.float().cpu().numpy(), want)
