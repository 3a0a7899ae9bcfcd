"""smd_paged4_append and smd_paged4_read on the GPU against the 64-bit oracle: the values that
the codes stand for, the scales and the bounds are equal, bit for bit."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import paged as opaged
from oracle import paged4 as opaged4
from paged4_common import Cache4
from paged_common import bf16, i32

pytestmark = pytest.mark.gpu


def check(cuda, cache, x, slots, fused=0, bounds=True):
    """Appends to a copy of the cache on the GPU and compares the whole pool, then reads the slots."""
    import torch
    from sparse_mla_decode_gb300 import binding
    gpu = cache.to(cuda, bounds)
    T, heads, D = x[0].shape
    k, v = bf16(x[0], cuda), bf16(x[1], cuda)
    if fused:  # tokens lie apart
        wide = torch.full((T, (2 * heads + fused) * D), float("nan"), dtype=torch.bfloat16, device=cuda)
        wide[:, :heads * D], wide[:, -heads * D:] = k.flatten(1), v.flatten(1)
        k, v = wide[:, :heads * D].view(T, heads, D), wide[:, -heads * D:].view(T, heads, D)
    s = i32(slots, cuda)
    binding.paged4_append(gpu, k, v, s)
    got = binding.paged4_read(gpu, s)
    torch.cuda.synchronize()
    pools, scales = [c.copy() for c in cache.codes], [c.copy() for c in cache.scales]
    b = cache.bounds.copy() if bounds else None
    opaged4.paged4_append(pools, scales, cache.exps, b, x, slots)
    live = (slots >= 0) & (slots // cache.P < cache.pages)
    for side, (t, ts, back) in enumerate(((gpu.k, gpu.k_scales, got[0]), (gpu.v, gpu.v_scales, got[1]))):
        nan = opaged.VALUES[scales[side]]
        assert np.array_equal(ts.cpu().numpy(), scales[side])
        want = opaged4.values(pools[side], scales[side], cache.exps[side])
        mine = opaged4.values(t.cpu().numpy(), scales[side], cache.exps[side])
        assert np.array_equal(mine, want, equal_nan=True), "codes"
        assert nan.shape == scales[side].shape
        rows = back.float().cpu().numpy().astype(np.float64)
        assert (rows[~live] == 0).all()
        at = slots[live]
        assert np.array_equal(rows[live], want[at // cache.P, :, at % cache.P], equal_nan=True), "read"
    if bounds:
        assert np.array_equal(gpu.bounds.float().cpu().numpy().astype(np.float64), b), "bounds"


def tokens(rng, T, heads, D):
    return [opaged.bf16_round(rng.standard_normal((T, heads, D)) * np.exp2(rng.integers(-5, 6, (T, heads, 1))))
            for _ in "kv"]


def runs(rng, P, pages, spans):
    """Slots of runs (page, offset, length) in pages of their own."""
    slots = []
    for page, (o, n) in zip(rng.permutation(pages), spans):
        slots += list(page * P + o + np.arange(n))
    return np.array(slots)


@pytest.mark.parametrize("D,P,heads,layout,fused,exps", [
    (128, 64, 2, "heads", 0, True), (64, 16, 5, "tokens", 3, True), (256, 48, 1, "paired", 0, False),
    (128, 256, 3, "tokens", 1, False), (64, 80, 8, "heads", 0, True), (256, 16, 4, "tokens", 2, True)])
@pytest.mark.parametrize("bounds", [True, False])
def test_runs_of_every_kind(cuda, D, P, heads, layout, fused, exps, bounds):
    rng = np.random.default_rng(D + P + heads)
    spans = [(0, 1), (0, P), (3, P - 3), (P - 1, 1), (5, 7), (0, 9), (1, 1), (2, 8)]
    slots = runs(rng, P, 12, spans)
    check(cuda, Cache4(1, 12, heads, P, D, layout, exps), tokens(rng, len(slots), heads, D), slots, fused, bounds)


@pytest.mark.parametrize("D,P,heads", [(128, 64, 8), (64, 16, 16), (256, 128, 4), (128, 256, 1)])
def test_many_tokens(cuda, D, P, heads):
    """Past the limit of the form for few tokens: runs cross its chunks, short and long."""
    rng = np.random.default_rng(D)
    pages = max(160 * 256 // heads // P, 1) + 60
    spans = [(0, P) if i % 3 else (int(o := rng.integers(0, P)), int(rng.integers(1, P - o + 1))) for i in range(pages)]
    slots = runs(rng, P, pages, spans)
    assert len(slots) * heads * 2 > 152 * 256
    cache = Cache4(2, pages, heads, P, D)
    check(cuda, cache, tokens(rng, len(slots), heads, D), slots)


@pytest.mark.parametrize("T", [1, 40, 3000])
def test_slots_that_are_skipped(cuda, T):
    rng = np.random.default_rng(T)
    P, pages, heads, D = 32, 110, 8, 64
    slots = rng.permutation(pages * P)[:T]  # any order: runs of one token, mostly
    slots = np.sort(slots)
    slots[rng.random(T) < 0.3] = -1
    slots[rng.random(T) < 0.1] = pages * P + 5
    # a page may be in one run of a call where bounds are kept
    check(cuda, Cache4(3, pages, heads, P, D), tokens(rng, T, heads, D), slots, bounds=False)


def test_borders_between_codes_and_scales(cuda):
    """Every value on a border between two codes, and next to it, for every scale that a block can
    have; block maxima on borders between scales. Random blocks of bf16 besides."""
    rng = np.random.default_rng(5)
    D, P, heads = 128, 256, 1
    rows = []
    step = 1 + 2.0 ** -7
    for e in range(-4, 5):
        for m in range(8, 16):
            top = 6 * m * 2.0 ** (e - 3)  # a block whose scale is m 2^(e - 3)
            s = m * 2.0 ** (e - 3)
            border = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]) * s
            for b in (border, -border, border * step, border / step):
                rows.append(np.concatenate([[top], b, [s / 8] * 8]))
    for b in (17, 19, 21, 23, 25, 27, 29, 31):  # maxima halfway between two scales
        for e in range(-6, 4):
            top = 6 * b * 2.0 ** (e - 4)
            for t in (top, top * step, top / step):
                rows.append(np.concatenate([[t], rng.uniform(-t, t, 15)]))
    for e in range(-14, -4):  # scales below the normal ones, and none
        rows += [np.concatenate([[6 * m * 2.0 ** (e - 3)], rng.uniform(-1, 1, 15) * 2.0 ** e]) for m in (1, 2, 3, 5, 7, 9)]
    rows = np.array(rows + list(rng.standard_normal((8 * 4000 - len(rows), 16)) * np.exp2(rng.integers(-8, 9, (8 * 4000 - len(rows), 1)))))
    x = opaged.bf16_round(rows.reshape(-1, heads, D))
    T = x.shape[0]
    cache = Cache4(4, -(-T // P), heads, P, D, exps=False)
    check(cuda, cache, [x, -x], np.arange(T))
    check(cuda, cache, [x[:300], x[300:600]], np.arange(300))


@pytest.mark.parametrize("many", [False, True])
def test_zeros_nans_infinities_and_extremes(cuda, many):
    rng = np.random.default_rng(6)
    D, P, heads = 64, 32, 3
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
    n = 300 if many else 1
    x = [np.concatenate([y] * n) for y in x]
    slots = np.arange(32 * n)
    for e in (False, True):
        cache = Cache4(7, n + 1, heads, P, D, exps=e)
        if e:
            cache.exps = [np.array([100, -100, 7]), np.array([-400, 60, 400])]
        check(cuda, cache, x, slots)


def test_a_token_changes_nothing_but_its_own_slot_and_may_be_written_again(cuda):
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(8)
    cache = Cache4(9, 3, 2, 32, 128)
    c = cache.to(cuda)
    before = [t.clone() for t in (c.k, c.v, c.k_scales, c.v_scales)]
    x = tokens(rng, 4, 2, 128)
    s = i32([40, 41, 42, 43], cuda)
    k, v = bf16(x[0], cuda), bf16(x[1], cuda)
    binding.paged4_append(c, k * 100, v * 100, s)  # drafts, of which the last two are rejected
    binding.paged4_append(c, k[:2], v[:2], s[2:])
    got = binding.paged4_read(c, s)
    one = binding.PagedCache4.empty(1, 2, 16, 128, bounds=False, k_exp=c.k_exp, v_exp=c.v_exp, device=cuda)
    binding.paged4_append(one, k[:2], v[:2], s[:2] - 40)
    want = binding.paged4_read(one, s[:2] - 40)
    for a, b in zip(got, want):
        assert torch.equal(a[2:], b)
    for t, was in zip((c.k, c.v, c.k_scales, c.v_scales), before):
        t, was = t.clone(), was.clone()
        t[1, :, 8:12] = was[1, :, 8:12] = 0
        assert torch.equal(t, was)


def test_reading_one_side_into_rows_that_lie_apart(cuda):
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(10)
    cache = Cache4(11, 6, 3, 16, 64, "tokens")
    c = cache.to(cuda)
    slots = np.array([5, 5, -1, 95, 96, 2 ** 31 - 1, 0])
    wide = torch.full((7, 8 * 64), 3.0, dtype=torch.bfloat16, device=cuda)
    k = wide[:, 64:4 * 64].view(7, 3, 64)
    binding.paged4_read(c, i32(slots, cuda), k=k, v=torch.empty_like(k.contiguous()))
    want = cache.values(0)
    got = wide.float().cpu().numpy()
    assert (got[:, :64] == 3).all() and (got[:, 256:] == 3).all()
    for t, s in enumerate(slots):
        row = want[s // 16, :, s % 16].reshape(-1) if 0 <= s < 96 else np.full(192, 3.0)
        assert np.array_equal(got[t, 64:256], row)
    so = binding.lib()
    out = torch.zeros((2, 3, 64), dtype=torch.bfloat16, device=cuda)
    s = i32([7, 20], cuda)
    assert so.smd_paged4_read(c.ref, s.data_ptr(), 2, 0, 0, out.data_ptr(), 192, torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert np.array_equal(out.float().cpu().numpy(), cache.values(1)[[0, 1], :, [7, 4]])


def test_a_pool_past_32_bit_offsets_and_a_graph(cuda):
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(12)
    P, D, heads = 64, 128, 8
    pages = 2 ** 32 // (P * D // 2 * heads) + 10
    c = binding.PagedCache4.empty(pages, heads, P, D, bounds=True, device=cuda)
    x = tokens(rng, 5, heads, D)
    slots = i32(pages * P - 5 + np.arange(5), cuda)
    k, v = bf16(x[0], cuda), bf16(x[1], cuda)
    out = [torch.zeros_like(k) for _ in "kv"]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        binding.paged4_append(c, k, v, slots)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.paged4_append(c, k, v, slots)
        binding.paged4_read(c, slots, *out)
    k.copy_(bf16(x[1], cuda))
    graph.replay()
    torch.cuda.synchronize()
    want = opaged4.quantise(x[1], np.zeros(heads))
    want = opaged4.VALUES[opaged4.unpack(want[0])].reshape(5, heads, -1, 16) * opaged.VALUES[want[1]][..., None]
    for t in out:
        assert np.array_equal(t.float().cpu().numpy().astype(np.float64), want.reshape(5, heads, D))
    assert int((c.k[:-1] != 0).sum()) == 0


@pytest.mark.parametrize("D,heads,T", [(64, 3, 40), (128, 9, 300), (256, 1, 700), (128, 17, 5)])
@pytest.mark.parametrize("off", [0, 8, 16, 24])
def test_rows_read_to_every_alignment(cuda, D, heads, T, off):
    """The same bits, and nothing beside the rows, whether rows lie 16 or 32 bytes apart from a sector."""
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(D + heads)
    cache = Cache4(8, -(-T // 32) + 1, heads, 32, D)
    c = cache.to(cuda)
    slots = rng.permutation(cache.pages * 32)[:T]
    slots[T // 2] = -1
    want = binding.paged4_read(c, i32(slots, cuda))
    row = heads * D
    for step in (row, row + 8, row + 16):
        flat = [torch.full((T * step + 32,), 3.0, dtype=torch.bfloat16, device=cuda) for _ in "kv"]
        out = [x[off:].as_strided((T, heads, D), (step, D, 1)) for x in flat]
        binding.paged4_read(c, i32(slots, cuda), *out)
        torch.cuda.synchronize()
        for x, o, w in zip(flat, out, want):
            keep = torch.ones(T, dtype=torch.bool, device=cuda)
            keep[T // 2] = False
            assert torch.equal(o[keep], w[keep]) and bool((o[~keep] == 3.0).all())
            o.fill_(3.0)
            assert bool((x == 3.0).all())
