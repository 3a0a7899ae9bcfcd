"""smd_paged_append on the GPU: codes, scales and bounds equal the oracle's,
value for value (every quotient by a power of two is exact)."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import paged as opaged
from paged_common import Cache, bf16, i32

pytestmark = pytest.mark.gpu


def check(cuda, cache, x, slots, fused=0):
    import torch
    from sparse_mla_decode_gb300 import binding
    c = cache.to(cuda)
    kv = [bf16(y, cuda) for y in x]
    if fused:  # slices of wider rows
        T, heads, D = kv[0].shape
        wide = torch.zeros((T, 2 * heads * D + fused), dtype=torch.bfloat16, device=cuda)
        wide[:, :heads * D] = kv[1].flatten(1)
        wide[:, -heads * D:] = kv[0].flatten(1)
        kv = [wide[:, -heads * D:].view(T, heads, D), wide[:, :heads * D].view(T, heads, D)]
    binding.paged_append(c, kv[0], kv[1], i32(slots, cuda))
    torch.cuda.synchronize()
    codes = [y.copy() for y in cache.codes]
    scales = [y.copy() for y in cache.scales]
    bounds = cache.bounds.copy()
    opaged.paged_append(codes, scales, bounds, x, slots)
    for side, got, gs in ((0, c.k, c.k_scale), (1, c.v, c.v_scale)):
        assert np.array_equal(gs.cpu().numpy(), scales[side]), "kv"[side] + " scales"
        want, have = codes[side], got.cpu().numpy()
        same = (have == want) | (((have & 127) == 127) & ((want & 127) == 127))
        assert same.all(), "kv"[side] + " codes"
    assert np.array_equal(c.bounds.float().cpu().numpy(), bounds.astype(np.float32)), "bounds"
    return c


def tokens(rng, T, heads, D):
    size = np.exp2(rng.integers(-6, 7, (T, heads, 1)))
    return [opaged.bf16_round(rng.standard_normal((T, heads, D)) * size) for _ in "kv"]


def runs(rng, P, pages, spans):
    """Slots of runs (offset, tokens) on distinct pages."""
    free = list(rng.permutation(pages))
    out = []
    for o, n in spans:
        page = free.pop()
        out += [page * P + o + i for i in range(n)]
    return np.array(out, dtype=np.int32)


@pytest.mark.parametrize("D,P,heads,layout,fused", [
    (128, 64, 2, "heads", 0), (128, 16, 3, "tokens", 8), (64, 48, 1, "paired", 0),
    (64, 128, 5, "tokens", 64), (256, 32, 2, "heads", 256), (128, 256, 1, "heads", 0),
    (256, 256, 1, "tokens", 0)])
def test_runs_of_every_kind(cuda, D, P, heads, layout, fused):
    """One token, pages filled whole, runs that begin or end inside a page."""
    rng = np.random.default_rng(D + P)
    spans = [(0, 1), (P - 1, 1), (0, P), (3, 1), (5, P - 5), (0, P - 1), (7, 4), (P // 2, 3), (1, 2)]
    slots = runs(rng, P, 12, spans)
    cache = Cache(1, 12, heads, P, D, layout)
    check(cuda, cache, tokens(rng, len(slots), heads, D), slots, fused)


@pytest.mark.parametrize("D,P,heads", [(128, 64, 8), (64, 16, 16), (256, 128, 4)])
def test_many_tokens(cuda, D, P, heads):
    """Prompts: enough tokens for blocks instead of warps; runs cross the blocks' chunks."""
    rng = np.random.default_rng(3)
    spans, T = [], 0
    while T < 5000:
        o = int(rng.integers(0, P)) if rng.random() < 0.3 else 0
        n = P - o if rng.random() < 0.7 else int(rng.integers(1, P - o + 1))
        spans.append((o, n))
        T += n
    slots = runs(rng, P, len(spans) + 2, spans)
    cache = Cache(2, len(spans) + 2, heads, P, D)
    check(cuda, cache, tokens(rng, len(slots), heads, D), slots)


@pytest.mark.parametrize("T", [1, 40, 4096])
def test_slots_that_are_skipped(cuda, T):
    """Negative slots and slots past the pool write nothing and end runs."""
    rng = np.random.default_rng(T)
    P, heads, D, pages = 32, 4, 128, T // 32 + 3
    slots = np.arange(T, dtype=np.int32) + 32
    slots[rng.random(T) < 0.2] = -1
    slots[rng.random(T) < 0.1] = pages * P + 3
    slots[0] = 2 ** 31 - 1 if T > 1 else -1
    # a skipped token splits a page's run: leave the page to the first part
    for t in range(1, T):
        if slots[t] >= 0 and slots[t] < pages * P and slots[t] % P and slots[t - 1] != slots[t] - 1:
            while t < T and slots[t] >= 0 and slots[t] % P:
                slots[t] = -7
                t += 1
    check(cuda, Cache(3, pages, heads, P, D), tokens(rng, T, heads, D), slots)


@pytest.mark.parametrize("many", [False, True])
def test_zeros_nans_infinities_and_extremes(cuda, many):
    rng = np.random.default_rng(6)
    P, heads, D = 32, 2 if not many else 32, 128
    reps = 1 if not many else 60
    spans = [(0, 3), (4, 2), (0, 1), (9, 5), (0, 4), (2, 1), (0, 2), (5, 1)] * reps
    slots = runs(rng, P, len(spans), spans)
    x = tokens(rng, len(slots), heads, D)
    cache = Cache(4, len(spans), heads, P, D)
    at = np.cumsum([0] + [n for _, n in spans])
    for i in range(0, len(spans), 8):
        s = [slice(at[i + j], at[i + j + 1]) for j in range(8)]
        for y in x:
            y[s[0]] = 0.0
            y[s[1], :, 3] = np.nan
            y[s[2]] = np.nan
            y[s[3], 0, 7] = np.inf
            y[s[3], 1, 9] = -np.inf
            y[s[4]] = opaged.bf16_round(y[s[4]] * 2.0 ** -120)
            y[s[5]] = opaged.bf16_round(y[s[5]] * 2.0 ** 110)
            y[s[6], :, :5] = [448.0, -450.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10]
            y[s[6], :, 5:] = 0.0
            y[s[7]] = -0.0
    check(cuda, cache, x, slots)


def test_kept_codes_move_with_the_scale(cuda):
    """A token far larger than the page's others: their codes are written again;
    one far smaller: nothing but the token is written; a page whose scale is no
    power of two keeps it while it is the larger."""
    rng = np.random.default_rng(8)
    P, heads, D = 64, 2, 128
    cache = Cache(5, 6, heads, P, D)
    cache.scales[0][4] = np.float32(0.3)
    cache.scales[1][4] = np.float32(1.7)
    cache.codes[0][2, :, 5, 9] = 0x7f  # a kept NaN stays one
    slots = np.array([1 * P + 20, 2 * P + 63, 3 * P + 1, 4 * P + 31], dtype=np.int32)
    x = tokens(rng, 4, heads, D)
    for y, size in zip(range(4), (2.0 ** 6, 2.0 ** 3, 2.0 ** -12, 2.0 ** -4)):
        for side in x:
            side[y] = opaged.bf16_round(rng.standard_normal((heads, D)) * size)
    c = check(cuda, cache, x, slots)
    assert np.float32(0.3) in c.k_scale[4].cpu().numpy()


def test_a_rejected_token_is_written_over(cuda):
    """The slot of a token that was not kept is given again: the page's tokens
    before it are kept, the token replaced."""
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(9)
    P, heads, D = 16, 1, 64
    cache = Cache(6, 3, heads, P, D)
    x = tokens(rng, 3, heads, D)
    first = np.array([P + 4, P + 5, P + 6], dtype=np.int32)
    c = check(cuda, cache, x, first)
    opaged.paged_append(cache.codes, cache.scales, cache.bounds, x, first)
    y = tokens(rng, 1, heads, D)
    binding.paged_append(c, bf16(y[0], cuda), bf16(y[1], cuda), i32([P + 5], cuda))
    torch.cuda.synchronize()
    opaged.paged_append(cache.codes, cache.scales, cache.bounds, y, np.array([P + 5]))
    assert np.array_equal(c.k.cpu().numpy(), cache.codes[0])
    assert np.array_equal(c.v_scale.cpu().numpy(), cache.scales[1])


def test_a_cache_without_bounds_and_refusals(cuda):
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(10)
    c = binding.PagedCache.empty(4, 2, 32, 128, bounds=False, device=cuda)
    x = tokens(rng, 3, 2, 128)
    k, v, slots = bf16(x[0], cuda), bf16(x[1], cuda), i32([0, 1, 40], cuda)
    binding.paged_append(c, k, v, slots)
    binding.paged_append(c, k[:0], v[:0], slots[:0])
    torch.cuda.synchronize()
    assert int((c.k_scale != 0).sum()) == 4
    with pytest.raises(ValueError):
        binding.paged_append(c, k.float(), v, slots)
    with pytest.raises(ValueError):
        binding.paged_append(c, k[:2], v, slots)
    odd = torch.zeros((3, 2 * 128 + 4), dtype=torch.bfloat16, device=cuda)[:, :256].view(3, 2, 128)
    with pytest.raises(binding.SmdError) as e:
        binding.paged_append(c, odd, v, slots)
    assert e.value.status == binding.SMD_ERR_SHAPE
    only = binding.PagedCache(bounds=torch.zeros((4, 2, 2, 128), dtype=torch.bfloat16, device=cuda),
                              page_size=32)
    with pytest.raises(binding.SmdError) as e:
        binding.paged_append(only, k, v, slots)
    assert e.value.status == binding.SMD_ERR_NULL
    with pytest.raises(ValueError):
        binding.PagedCache(c.k, c.v[:, :1], c.k_scale, c.v_scale)
    with pytest.raises(binding.SmdError) as e:
        binding.PagedCache(c.k[:, :, :24], c.v[:, :, :24], c.k_scale, c.v_scale)
    assert e.value.status == binding.SMD_ERR_SHAPE
