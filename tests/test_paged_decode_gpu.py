"""smd_paged_decode on the GPU against the 64-bit oracle (tolerances:
paged_common.tolerances)."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import paged as opaged
from paged_common import Cache, bf16, check_decode, i32, table_for

pytestmark = pytest.mark.gpu


def queries(rng, B, Hq, D, size=1.0):
    return opaged.bf16_round(rng.standard_normal((B, Hq, D)) * size)


def run(cuda, cache, q, table, lengths, G=1, lists=None, counts=None, gpu_cache=None, **kw):
    import torch
    from sparse_mla_decode_gb300 import binding
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    ws = torch.zeros(binding.paged_workspace_bytes(gpu_cache or cache.to(cuda)), dtype=torch.uint8,
                     device=cuda)
    out, lse = binding.paged_decode(
        bf16(q, cuda), gpu_cache or cache.to(cuda), i32(table, cuda), i32(lengths, cuda),
        cache.D ** -0.5, row_group=G, block_lists=None if lists is None else i32(lists, cuda),
        block_counts=None if counts is None else i32(counts, cuda), status=status, workspace=ws, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return out, lse


def oracle(cache, q, table, lengths, G=1, lists=None, counts=None):
    return opaged.paged_decode(q, cache.codes, cache.scales, table, lengths, cache.D ** -0.5, G,
                               lists, counts)


LENGTHS = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 250, 500, 777]


@pytest.mark.parametrize("D,P,heads,g,G,layout", [
    (128, 64, 2, 8, 1, "heads"), (128, 64, 3, 1, 1, "tokens"), (128, 16, 2, 4, 1, "heads"),
    (128, 48, 1, 16, 1, "tokens"), (128, 32, 2, 7, 4, "heads"), (128, 128, 1, 16, 2, "paired"),
    (128, 80, 2, 17, 1, "heads"), (128, 64, 1, 40, 3, "heads"), (128, 256, 1, 3, 8, "tokens"),
    (64, 16, 5, 3, 4, "tokens"), (64, 64, 2, 8, 1, "paired"), (64, 48, 2, 12, 2, "heads"),
    (64, 32, 1, 33, 1, "heads"), (256, 16, 2, 4, 1, "heads"), (256, 64, 1, 8, 2, "tokens"),
    (256, 32, 1, 20, 1, "paired"), (128, 64, 1, 128, 1, "heads")])
def test_lengths_layouts_and_groups(cuda, D, P, heads, g, G, layout):
    rng = np.random.default_rng(D + P + g)
    pages = sum(-(-n // P) for n in LENGTHS) + 3
    cache = Cache(1, pages, heads, P, D, layout)
    table = table_for(rng, LENGTHS, P, pages, extra=2)
    q = queries(rng, len(LENGTHS) * G, heads * g, D, 2.0)
    got = run(cuda, cache, q, table, LENGTHS, G)
    check_decode(*got, oracle(cache, q, table, LENGTHS, G), f"{D} {P} {heads} {g} {G}")


@pytest.mark.parametrize("D,P,g,lengths", [(128, 64, 8, [9000, 3, 70]), (64, 16, 4, [6001]),
                                           (256, 32, 2, [4097, 4096]), (128, 128, 16, [20000])])
def test_long_rows_are_cut_over_the_grid_and_joined(cuda, D, P, g, lengths):
    import torch
    rng = np.random.default_rng(5)
    pages = sum(-(-n // P) for n in lengths) + 1
    cache = Cache(2, pages, 2, P, D)
    table = table_for(rng, lengths, P, pages)
    q = queries(rng, len(lengths), 2 * g, D, 3.0)
    got = run(cuda, cache, q, table, lengths)
    check_decode(*got, oracle(cache, q, table, lengths), f"{D} {lengths}")
    again = run(cuda, cache, q, table, lengths)
    assert torch.equal(got[0].view(torch.int16), again[0].view(torch.int16))
    assert torch.equal(got[1], again[1])


@pytest.mark.parametrize("P", [16, 48, 64])
def test_one_dominant_token_at_every_place_gives_its_values(cuda, P):
    """A token whose logit exceeds the others' by more than 2^-24 allows is the
    row's output: the page, the offset and the token's place in it are right."""
    D, n = 128, 3 * P + 5
    rng = np.random.default_rng(P)
    cache = Cache(3, n * 5, 1, P, D)
    lengths = [n] * n
    table = table_for(rng, lengths, P, n * 5)
    q = queries(rng, n, 2, D)
    for r in range(n):
        p, o = table[r, r // P], r % P
        cache.codes[0][p, 0, o] = opaged.e4m3_encode(q[r, 0] * 200)
        cache.scales[0][table[r, :4], 0] = 2.0 ** -3
    q[:, 1] = q[:, 0]
    out, lse = run(cuda, cache, q, table, lengths)
    k = cache.values(0)
    for r in range(n):  # it dominates
        s = np.concatenate(k[table[r, :-(-n // P)], 0])[:n] @ q[r, 0] * D ** -0.5
        assert s.argmax() == r and s[r] - np.delete(s, r).max() > 24 * np.log(2)
    check_decode(out, lse, oracle(cache, q, table, lengths))


@pytest.mark.parametrize("D,G", [(64, 4), (128, 1), (128, 3), (256, 2)])
def test_codes_that_no_row_sees_do_not_matter(cuda, D, G):
    """NaN codes past the lengths, in unused pages, and in a verify token that
    only the later rows see; scales of unused pages are infinite."""
    rng = np.random.default_rng(7)
    P, g, heads = 64, 3, 2
    lengths = [0, 1, 5, 64, 65, 100, 190]
    pages = 12
    cache = Cache(4, pages, heads, P, D)
    table = table_for(rng, lengths, P, pages)
    held = np.zeros((pages, P), dtype=bool)
    for r, n in enumerate(lengths):
        for t in range(n):
            held[table[r, t // P], t % P] = True
    for c in cache.codes:
        c[np.broadcast_to(~held[:, None, :, None], c.shape)] = 0x7f
        c[..., 3][~np.broadcast_to(held[:, None], c.shape[:3])] = 0xff
    for s in cache.scales:
        s[~held.any(1)] = np.inf
    if G > 1:  # the last token of request 5, in one column
        cache.codes[1][table[5, 1], :, 99 - P, 17] = 0x7f
        cache.codes[0][table[4, 1], :, 64 - P, 5] = 0xff  # a key: its whole rows
    q = queries(rng, len(lengths) * G, heads * g, D)
    ref = oracle(cache, q, table, lengths, G)
    if G > 1:
        nan = np.isnan(ref[0])
        assert nan[5 * G + G - 1, :, 17].all() and nan[5 * G + G - 1].sum() == heads * g
        assert not nan[5 * G:5 * G + G - 1].any()
        assert nan[4 * G + G - 1].all() and not nan[4 * G:4 * G + G - 1].any()
        bad = np.isnan(ref[1])
        out, lse = run(cuda, cache, q, table, lengths, G)
        assert np.array_equal(np.isnan(lse.cpu().numpy()), bad)
        keep = ~bad.any(1)
        check_decode(out[keep.tolist()], lse[keep.tolist()], tuple(x[keep] for x in ref))
        assert np.isnan(out.float().cpu().numpy()[~keep]).all()
    else:
        check_decode(*run(cuda, cache, q, table, lengths, G), ref)


@pytest.mark.parametrize("D,P,g,G", [(128, 64, 4, 1), (128, 16, 8, 2), (64, 48, 20, 1), (256, 32, 4, 3)])
def test_lists_of_pages(cuda, D, P, g, G):
    """Any order, duplicates, pages past the row's end, -1, empty lists, counts
    below and beyond the width."""
    rng = np.random.default_rng(11)
    lengths = [700, 1, 0, 333, P, 3 * P + 1]
    heads, K = 2, 9
    pages = sum(-(-n // P) for n in lengths) + 1
    cache = Cache(5, pages, heads, P, D)
    table = table_for(rng, lengths, P, pages)
    B = len(lengths) * G
    lists = rng.integers(-2, max(lengths) // P + 3, (B, heads, K))
    lists[0, 0] = 0                     # one page nine times
    counts = rng.integers(0, K + 1, (B, heads))
    counts[0, 0], counts[-1, 0], counts[-1, 1] = K + 5, -3, 0
    q = queries(rng, B, heads * g, D, 2.0)
    ref = oracle(cache, q, table, lengths, G, lists, counts)
    check_decode(*run(cuda, cache, q, table, lengths, G, lists, counts), ref)
    ref = oracle(cache, q, table, lengths, G, lists)
    check_decode(*run(cuda, cache, q, table, lengths, G, lists), ref, "no counts")
    out, lse = run(cuda, cache, q, table, lengths, G, lists[:, :, :0])
    assert (out == 0).all() and np.isneginf(lse.cpu().numpy()).all()


def test_lists_of_every_page_are_the_whole_row(cuda):
    rng = np.random.default_rng(12)
    P, D, lengths = 64, 128, [1000, 64, 200]
    pages = 30
    cache = Cache(6, pages, 2, P, D)
    table = table_for(rng, lengths, P, pages)
    q = queries(rng, 3, 8, D, 2.0)
    lists = np.broadcast_to(np.arange(table.shape[1]), (3, 2, table.shape[1]))
    ref = oracle(cache, q, table, lengths)
    check_decode(*run(cuda, cache, q, table, lengths, lists=lists), ref)


def test_scales_and_query_sizes_over_the_range_of_floats(cuda):
    """Scales from 2^-60 to 2^60 within one row, a zero query row, rows of 2^-60
    and 2^30, heads of very different size."""
    rng = np.random.default_rng(13)
    P, D, lengths = 32, 128, [150, 150, 150, 150]
    pages = 24
    cache = Cache(7, pages, 1, P, D)
    table = table_for(rng, lengths, P, pages)
    for r in range(4):
        for j in range(5):
            cache.scales[1][table[r, j]] = 2.0 ** [-60, 3, -2, 60, 40][j] if r < 2 else 2.0 ** (j - 9)
    cache.scales[0][table[0, :5]] = 2.0 ** 50
    cache.scales[1][table[1, 3:5]] = 1.5 * 2.0 ** -7  # no power of two
    q = queries(rng, 4, 4, D)
    q[0] = opaged.bf16_round(q[0] * 2.0 ** -56)
    q[1, 0] = 0.0
    q[1, 1] = opaged.bf16_round(q[1, 1] * 2.0 ** -60)
    q[2, :, ::2] = opaged.bf16_round(q[2, :, ::2] * 2.0 ** -20)
    q[3, 0] = opaged.bf16_round(q[3, 0] * 16)
    check_decode(*run(cuda, cache, q, table, lengths), oracle(cache, q, table, lengths))


def test_more_requests_than_one_launch_takes(cuda):
    rng = np.random.default_rng(14)
    P, D = 16, 64
    lengths = rng.integers(0, 40, 2100)
    pages = int(sum(-(-n // P) for n in lengths)) + 1
    cache = Cache(8, pages, 1, P, D)
    table = table_for(rng, lengths, P, pages)
    q = queries(rng, len(lengths), 2, D, 2.0)
    check_decode(*run(cuda, cache, q, table, lengths), oracle(cache, q, table, lengths))


def test_table_entries_outside_the_pool_read_nothing(cuda):
    rng = np.random.default_rng(15)
    P, D, lengths = 32, 128, [100, 60]
    cache = Cache(9, 8, 2, P, D)
    table = table_for(rng, lengths, P, 8)
    table[0, 1], table[0, 3], table[1, 0] = -5, 8, 2 ** 31 - 1
    q = queries(rng, 2, 4, D)
    check_decode(*run(cuda, cache, q, table, lengths), oracle(cache, q, table, lengths))


def test_lengths_beyond_the_table_are_clamped(cuda):
    rng = np.random.default_rng(16)
    P, D = 32, 128
    cache = Cache(10, 8, 1, P, D)
    table = table_for(rng, [64, 64], P, 8)
    q = queries(rng, 2, 4, D)
    want = oracle(cache, q, table, [64, 0])
    check_decode(*run(cuda, cache, q, table, [5000, -7]), want)


def test_strided_queries_and_table_rows(cuda):
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(17)
    P, D, heads, g, lengths = 32, 128, 2, 3, [90, 33, 0, 1]
    cache = Cache(11, 12, heads, P, D)
    table = table_for(rng, lengths, P, 12)
    q = queries(rng, 4, heads * g, D)
    fused = torch.full((4, (heads * g + 4) * D), float("nan"), dtype=torch.bfloat16, device=cuda)
    fused[:, 2 * D:(2 + heads * g) * D] = bf16(q, cuda).flatten(1)
    wide = torch.full((4, table.shape[1] + 3), -1, dtype=torch.int32, device=cuda)
    wide[:, :table.shape[1]] = i32(table, cuda)
    out, lse = binding.paged_decode(
        fused[:, 2 * D:(2 + heads * g) * D].view(4, heads * g, D), cache.to(cuda),
        wide[:, :table.shape[1]], i32(lengths, cuda), D ** -0.5)
    check_decode(out, lse, oracle(cache, q, table, lengths))


def test_a_pool_past_32_bit_offsets(cuda):
    """Pages whose bytes lie beyond 2^32 in each side of the pool."""
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(18)
    P, D, heads = 64, 128, 8
    pages = 2 ** 32 // (P * D * heads) + 200
    small = Cache(12, 40, heads, P, D)
    pools = [torch.empty((pages, heads, P, D), dtype=torch.uint8, device=cuda) for _ in "kv"]
    scales = [torch.zeros((pages, heads), dtype=torch.float32, device=cuda) for _ in "kv"]
    where = np.concatenate([np.arange(20), pages - 1 - np.arange(20)])
    at = torch.from_numpy(where).to(cuda)
    for side in (0, 1):
        pools[side][at] = torch.from_numpy(small.codes[side]).to(cuda)
        scales[side][at] = torch.from_numpy(small.scales[side]).to(cuda)
    lengths = [1200, 1100]
    table = table_for(rng, lengths, P, 40)
    q = queries(rng, 2, heads * 4, D, 2.0)
    used = table < 40
    far = np.where(used, where[np.where(used, table, 0)], -1)
    cache = binding.PagedCache(*pools, *scales)
    out, lse = binding.paged_decode(bf16(q, cuda), cache, i32(far, cuda), i32(lengths, cuda), D ** -0.5)
    check_decode(out, lse, oracle(small, q, table, lengths))


def test_another_stream_and_a_graph_give_the_same_bits(cuda):
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(19)
    P, D, lengths = 64, 128, [3000, 17, 0]
    cache = Cache(13, 60, 2, P, D)
    table = table_for(rng, [3000, 17, 100], P, 60)
    q = queries(rng, 3, 8, D)
    c, tq, tt, tl = cache.to(cuda), bf16(q, cuda), i32(table, cuda), i32(lengths, cuda)
    ws = torch.zeros(binding.paged_workspace_bytes(c), dtype=torch.uint8, device=cuda)
    out, lse = binding.paged_decode(tq, c, tt, tl, D ** -0.5, workspace=ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out2, lse2 = torch.zeros_like(out), torch.zeros_like(lse)
    with torch.cuda.stream(side):
        binding.paged_decode(tq, c, tt, tl, D ** -0.5, workspace=ws, out=out2, lse=lse2)
    side.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    graph = torch.cuda.CUDAGraph()
    out3, lse3 = torch.zeros_like(out), torch.zeros_like(lse)
    with torch.cuda.graph(graph):
        binding.paged_decode(tq, c, tt, tl, D ** -0.5, workspace=ws, out=out3, lse=lse3)
    tl[2] = 100  # a replay goes by what the buffers hold then
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    check_decode(out3, lse3, oracle(cache, q, table, [3000, 17, 100]))


def test_nothing_to_do_and_refusals(cuda):
    import torch
    from sparse_mla_decode_gb300 import binding
    cache = Cache(14, 4, 2, 32, 128)
    c = cache.to(cuda)
    none = binding.paged_decode(torch.empty((0, 4, 128), dtype=torch.bfloat16, device=cuda), c,
                                torch.empty((0, 2), dtype=torch.int32, device=cuda),
                                torch.empty(0, dtype=torch.int32, device=cuda), 0.1)
    assert none[0].shape == (0, 4, 128)
    q, t, n = bf16(np.zeros((2, 4, 128)), cuda), i32([[0, 1], [2, 3]], cuda), i32([3, 4], cuda)
    ws = torch.empty(binding.paged_workspace_bytes(c), dtype=torch.uint8, device=cuda)

    def status(**kw):
        with pytest.raises(binding.SmdError) as e:
            binding.paged_decode(kw.get("q", q), kw.get("c", c), t, n, 0.1,
                                 row_group=kw.get("G", 1), workspace=kw.get("ws", ws))
        return e.value.status

    assert status(ws=ws[:-16]) == binding.SMD_ERR_WORKSPACE
    assert status(ws=ws[4:]) == binding.SMD_ERR_WORKSPACE
    assert status(q=bf16(np.zeros((2, 3, 128)), cuda)) == binding.SMD_ERR_SHAPE  # 3 heads over 2
    assert status(q=bf16(np.zeros((18, 4, 128)), cuda), G=9) == binding.SMD_ERR_SHAPE
    only = binding.PagedCache(bounds=c.bounds, page_size=32)
    assert status(c=only) == binding.SMD_ERR_NULL
    with pytest.raises(ValueError):
        binding.paged_decode(q[:1], c, t, n, 0.1)
    with pytest.raises(ValueError):
        binding.paged_decode(q.float(), c, t, n, 0.1)
    with pytest.raises(ValueError):
        binding.paged_decode(q, c, t, n, 0.1, block_counts=n)


@pytest.mark.parametrize("D,P,g,G", [(64, 16, 8, 1), (64, 112, 5, 1), (64, 16, 20, 1), (64, 256, 24, 1),
                                     (128, 16, 6, 3), (128, 16, 20, 1), (256, 48, 9, 1)])
def test_tiles_of_one_page_and_of_two_with_and_without_lists(cuda, D, P, g, G):
    rng = np.random.default_rng(7 * D + P + g)
    lengths = [1, 40, 333, 1500]
    pages = sum(-(-n // P) for n in lengths) + 2
    cache = Cache(3, pages, 2, P, D)
    table = table_for(rng, lengths, P, pages, extra=1)
    q = queries(rng, len(lengths) * G, 2 * g, D, 2.0)
    check_decode(*run(cuda, cache, q, table, lengths, G), oracle(cache, q, table, lengths, G))
    K = 5
    lists = rng.integers(-1, max(-(-1500 // P), 2), (len(lengths) * G, 2, K))
    check_decode(*run(cuda, cache, q, table, lengths, G, lists),
                 oracle(cache, q, table, lengths, G, lists))


def test_scales_that_are_no_powers_of_two_and_far_apart(cuda):
    rng = np.random.default_rng(23)
    cache = Cache(4, 40, 2, 32, 128)
    cache.scales = [s * np.float32(2.0) ** rng.integers(-12, 13, s.shape) * rng.uniform(1, 2, s.shape)
                    for s in cache.scales]
    cache.scales = [s.astype(np.float32) for s in cache.scales]
    table = table_for(rng, [700, 90], 32, 40)
    q = queries(rng, 2, 8, 128, 2.0 ** -9)
    check_decode(*run(cuda, cache, q, table, [700, 90]), oracle(cache, q, table, [700, 90]))


def test_lists_for_more_heads_than_a_launch_takes_are_refused(cuda):
    import torch
    from sparse_mla_decode_gb300 import binding
    c = binding.PagedCache.empty(1, 130, 16, 64, bounds=False, device=cuda)
    t, n = i32([[0]], cuda), i32([16], cuda)
    ws = torch.zeros(binding.paged_workspace_bytes(c), dtype=torch.uint8, device=cuda)
    for G, fits in ((7, True), (8, False)):
        q = torch.zeros((G, 130, 64), dtype=torch.bfloat16, device=cuda)
        lists = torch.zeros((G, 130, 1), dtype=torch.int32, device=cuda)
        if fits:
            binding.paged_decode(q, c, t, n, 0.1, row_group=G, block_lists=lists, workspace=ws)
            continue
        with pytest.raises(binding.SmdError) as e:
            binding.paged_decode(q, c, t, n, 0.1, row_group=G, block_lists=lists, workspace=ws)
        assert e.value.status == binding.SMD_ERR_SHAPE
        binding.paged_decode(q, c, t, n, 0.1, row_group=G, workspace=ws)
    torch.cuda.synchronize()


@pytest.mark.parametrize("raw", [False, True])
def test_what_a_call_allocates_is_made_on_its_stream(cuda, raw):
    """The workspace is zeroed in the order of the call's stream, not behind what
    the current stream still has to do, and in memory that held something else."""
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(31)
    cache = Cache(5, 70, 2, 64, 128)
    c = cache.to(cuda)
    table = table_for(rng, [4000], 64, 70)
    q = queries(rng, 1, 16, 128)
    tq, tt, tl = bf16(q, cuda), i32(table, cuda), i32([4000], cuda)
    s = torch.cuda.Stream()
    used = torch.full((binding.paged_workspace_bytes(c),), 7, dtype=torch.uint8, device=cuda)
    torch.cuda.synchronize()
    del used
    torch.cuda._sleep(20_000_000)
    out, lse = binding.paged_decode(tq, c, tt, tl, 128 ** -0.5, stream=s.cuda_stream if raw else s)
    s.synchronize()
    got = out.cpu(), lse.cpu()
    torch.cuda.synchronize()
    check_decode(*got, oracle(cache, q, table, [4000]))


@pytest.mark.parametrize("D,P,g,G,stall", [
    (128, 64, 8, 1, 1), (128, 64, 8, 1, 4), (128, 16, 12, 2, 3), (128, 32, 32, 1, 2), (128, 48, 7, 4, 6),
    (64, 16, 3, 4, 6), (64, 64, 30, 1, 5), (256, 32, 4, 1, 3), (256, 64, 16, 1, 2)])
def test_a_wait_that_runs_out_gives_nan_rows_and_the_context_survives(cuda, D, P, g, G, stall):
    """The copy of every warp's tile number `stall` never completes. Each row is right or NaN
    throughout, the status says so, and the next call is right."""
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(D + P + stall)
    lengths = [200000, 0, 1, 40, 3000] + [int(n) for n in rng.integers(0, 700, 120)]
    cache = Cache(6, 80, 2, P, D)
    table = rng.integers(0, 80, (len(lengths), -(-200000 // P)))  # a range of 9 tiles or more for a warp
    q = queries(rng, len(lengths) * G, 2 * g, D, 2.0)
    ref = oracle(cache, q, table, lengths, G)
    c = cache.to(cuda)
    args = (bf16(q, cuda), c, i32(table, cuda), i32(lengths, cuda), D ** -0.5)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    ws = torch.zeros(binding.paged_workspace_bytes(c), dtype=torch.uint8, device=cuda)
    for with_status in (status, None):
        out, lse = binding.paged_decode(*args, row_group=G, status=with_status, workspace=ws,
                                        plan=dict(wait_budget_us=2000, inject_stall=stall))
        torch.cuda.synchronize()
        bad = np.isnan(lse.cpu().numpy())
        assert np.array_equal(np.isnan(out.float().cpu().numpy()), np.broadcast_to(bad[..., None], out.shape))
        assert bad.any() and (stall == 1) == bool(bad.all())
        good = torch.from_numpy(~bad)
        if not bad.all():
            check_decode(out.cpu()[good], lse.cpu()[good], tuple(x[~bad] for x in ref), "rows not stalled")
        ws.zero_()
    assert int(status.item()) == binding.SMD_ERR_TIMEOUT
    out, lse = binding.paged_decode(*args, row_group=G, workspace=ws)
    check_decode(out, lse, ref, "after a wait that ran out")


@pytest.mark.parametrize("D,P,g", [(64, 16, 3), (64, 32, 8), (128, 64, 8), (128, 48, 20), (256, 32, 4)])
def test_a_listed_page_that_only_a_later_verify_row_sees_does_not_matter(cuda, D, P, g):
    """Its values' scale is far above the others', it comes first in every row's list."""
    rng = np.random.default_rng(D + P)
    G, lengths = 2, [4 * P + 1, 5 * P + 1]
    cache = Cache(7, 20, 2, P, D)
    table = table_for(rng, lengths, P, 20)
    for r, n in enumerate(lengths):
        cache.scales[1][table[r, (n - 1) // P]] = 2.0 ** 60  # of the last token alone, which row 1 sees
    q = queries(rng, len(lengths) * G, 2 * g, D, 2.0)
    lists = np.tile(np.array([[4, 0, 2, 1], [5, 0, 3, 1]]).repeat(G, 0)[:, None], (1, 2, 1))
    ref = oracle(cache, q, table, lengths, G, lists)
    check_decode(*run(cuda, cache, q, table, lengths, G, lists), ref)


@pytest.mark.parametrize("D,P,g,G,n", [(64, 16, 3, 2, 49), (64, 48, 8, 3, 146), (128, 16, 8, 4, 18),
                                       (128, 80, 16, 2, 81), (128, 48, 12, 2, 241), (128, 64, 8, 2, 65),
                                       (256, 16, 4, 2, 33)])
def test_a_page_that_only_a_later_verify_row_sees_does_not_matter(cuda, D, P, g, G, n):
    """The values of a draft token that begins a page are far above the others' (or infinite: 2^120 is
    the scale that they are written with): the rows before it are as without it."""
    for scale in (2.0 ** 60, 2.0 ** 120):
        rng = np.random.default_rng(D + P)
        lengths = [n, 3 * n]
        cache = Cache(7, 60, 2, P, D)
        table = table_for(rng, lengths, P, 60)
        last = (n - 1) // P
        cache.scales[1][table[0, last]] = scale
        q = queries(rng, 2 * G, 2 * g, D, 2.0)
        ref = oracle(cache, q, table, lengths, G)
        seen = n - G + 1 + np.arange(G) > last * P
        assert seen.any() and not seen.all()
        out, lse = run(cuda, cache, q, table, lengths, G)
        rows = np.concatenate([~seen, np.ones(G, dtype=bool)])
        if scale == 2.0 ** 60:  # the rows that see it, too
            rows[:] = True
        check_decode(out.cpu()[rows], lse.cpu()[rows], tuple(x[rows] for x in ref), f"scale {scale}")


@pytest.mark.parametrize("D,P,G", [(64, 16, 1), (64, 32, 2), (128, 64, 1), (256, 16, 1)])
def test_requests_of_nearly_2_to_the_31_tokens(cuda, D, P, G):
    """As long as the table allows. All pages but a few lie outside the pool, so their tokens count as
    zeros: logits of 0 and no values."""
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(D + P)
    width = 2 ** 31 // P - 1
    cache = Cache(8, 6, 1, P, D)
    at = [0, 5, 2 ** 30 // P, width // 2, width - 2, width - 1]
    table = torch.full((1, width), -1, dtype=torch.int32, device=cuda)
    table[0, at] = torch.arange(6, dtype=torch.int32, device=cuda)
    q = queries(rng, G, 1, D)
    k, v = cache.values(0)[:, 0], cache.values(1)[:, 0]  # [6, P, D]
    for row in range(6):  # a token of each page at a logit of about 24, where 2^31 zeros weigh 8 %
        o = 3 * row % P if row < 5 else P - 1
        code = q[G - 1, 0] * (24 * D ** 0.5 / (q[G - 1, 0] ** 2).sum())
        cache.scales[0][row] = 2.0 ** -6
        cache.codes[0][row, 0, o] = opaged.e4m3_encode(code * 64)
        k[row] = opaged.VALUES[cache.codes[0][row, 0]] * 2.0 ** -6
    c = cache.to(cuda)
    for n in (width * P, width * P - 1, width * P - P + 1):
        out, lse = binding.paged_decode(bf16(q, cuda), c, table, i32([n], cuda), D ** -0.5, row_group=G)
        for i in range(G):
            lim = n - G + 1 + i
            seen = [min(max(lim - j * P, 0), P) for j in at]
            ks = np.concatenate([k[r, :m] for r, m in enumerate(seen)])
            vs = np.concatenate([v[r, :m] for r, m in enumerate(seen)])
            s = ks @ q[i, 0] * D ** -0.5
            total = np.exp(s).sum() + (lim - len(s))
            ref = (np.exp(s) @ vs / total)[None, None]
            reach = np.array([[D ** -0.5 * (np.abs(ks) @ np.abs(q[i, 0])).max()]])
            check_decode(out[i:i + 1], lse[i:i + 1], (ref, np.array([[np.log(total)]]), reach,
                                                      np.abs(vs).max(0)[None, None]), f"{n} {i}")


@pytest.mark.parametrize("D,P", [(64, 16), (128, 32), (256, 48)])
def test_lists_of_a_request_past_2_to_the_30_tokens(cuda, D, P):
    """Listed pages that the row does not have are passed over there, too."""
    rng = np.random.default_rng(D)
    n = 2 ** 30 + 5 * P + 3
    width = n // P + 3
    cache = Cache(9, 6, 2, P, D)
    table = np.full((1, width), -1, dtype=np.int32)
    last = (n - 1) // P
    at = [0, 1, last - 1, last]
    table[0, at] = [3, 0, 5, 1]
    lists = np.array([[[last, -1, width + 5, 0, last + 1, last + 2, -7], [-1, last - 1, -1, 1, -1, last + 1, 0]]])
    q = queries(rng, 1, 6, D)
    ref = oracle(cache, q, table, [n], 1, lists)
    check_decode(*run(cuda, cache, q, table, [n], 1, lists), ref)
