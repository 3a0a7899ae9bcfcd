"""smd_paged4_decode on the GPU against the 64-bit oracle (tolerances:
paged_common.tolerances; codes times block scales are exact in f16, as E4M3 codes are)."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import paged as opaged
from oracle import paged4 as opaged4
from paged4_common import Cache4
from paged_common import bf16, check_decode, i32, table_for

pytestmark = pytest.mark.gpu


def queries(rng, B, Hq, D, size=1.0):
    return opaged.bf16_round(rng.standard_normal((B, Hq, D)) * size)


def run(cuda, cache, q, table, lengths, G=1, lists=None, counts=None, gpu_cache=None, sm_scale=None, **kw):
    import torch
    from sparse_mla_decode_gb300 import binding
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    c = gpu_cache or cache.to(cuda)
    ws = torch.zeros(binding.paged4_workspace_bytes(c), dtype=torch.uint8, device=cuda)
    out, lse = binding.paged4_decode(
        bf16(q, cuda), c, i32(table, cuda), i32(lengths, cuda), cache.D ** -0.5 if sm_scale is None else sm_scale,
        row_group=G, block_lists=None if lists is None else i32(lists, cuda),
        block_counts=None if counts is None else i32(counts, cuda), status=status, workspace=ws, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return out, lse


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
    cache = Cache4(1, pages, heads, P, D, layout, exps=g % 2 == 0)
    table = table_for(rng, LENGTHS, P, pages, extra=2)
    q = queries(rng, len(LENGTHS) * G, heads * g, D)
    check_decode(*run(cuda, cache, q, table, LENGTHS, G), cache.attend(q, table, LENGTHS, G), f"{D} {P} {heads} {g} {G}")


@pytest.mark.parametrize("D,P,g,lengths", [(128, 64, 8, [9000, 3, 70]), (64, 16, 4, [6001]),
                                           (256, 32, 2, [4097, 4096]), (128, 128, 16, [20000])])
def test_long_rows_are_cut_over_the_grid_and_joined(cuda, D, P, g, lengths):
    import torch
    rng = np.random.default_rng(5)
    pages = sum(-(-n // P) for n in lengths) + 1
    cache = Cache4(2, pages, 2, P, D)
    table = table_for(rng, lengths, P, pages)
    q = queries(rng, len(lengths), 2 * g, D)
    got = run(cuda, cache, q, table, lengths)
    check_decode(*got, cache.attend(q, table, lengths), f"{D} {lengths}")
    again = run(cuda, cache, q, table, lengths)
    assert torch.equal(got[0].view(torch.int16), again[0].view(torch.int16))
    assert torch.equal(got[1], again[1])


@pytest.mark.parametrize("D,P", [(64, 16), (64, 64), (128, 16), (128, 48), (128, 64), (256, 32)])
def test_one_dominant_token_and_column_at_every_place(cuda, D, P):
    """Every token in turn outweighs the others by more than 2^-24 allows, by one column's block of
    its key: the row's output is its values. Page, offset, the token's place in a tile, the columns'
    order and the blocks' scales are right."""
    n = 3 * P + 5
    rng = np.random.default_rng(P)
    cache = Cache4(3, n * 5, 1, P, D, exps=False)
    lengths = [n] * n
    table = table_for(rng, lengths, P, n * 5)
    q = np.zeros((n, 2, D))
    for r in range(n):
        p, o, c = table[r, r // P], r % P, r * 7 % D
        q[r, :, c] = 32.0  # the only column of the logits
        for j in range(-(-n // P)):
            k = cache.codes[0][table[r, j], 0]
            k[:, c // 2] &= 0xf0 if c % 2 == 0 else 0x0f
        cache.codes[0][p, 0, o, c // 2] |= 7 if c % 2 == 0 else 0x70
        cache.scales[0][p, 0, o, c // 16] = opaged.e4m3_encode(np.array([12.0]))[0]
    out, lse = run(cuda, cache, q, table, lengths)
    assert 32 * 6 * 12 * D ** -0.5 > 24 * np.log(2)
    check_decode(out, lse, cache.attend(q, table, lengths))
    v = cache.values(1)
    want = np.stack([v[table[r, r // P], 0, r % P] for r in range(n)])
    assert np.array_equal(out[:, 0].float().cpu().numpy(), want)  # bf16 holds a value exactly


@pytest.mark.parametrize("D,G", [(64, 4), (128, 1), (128, 3), (256, 2)])
def test_scales_that_no_row_sees_do_not_matter(cuda, D, G):
    """NaN scales past the lengths, in unused pages, and in a verify token that only the later rows see."""
    rng = np.random.default_rng(7)
    P, g, heads = 64, 3, 2
    lengths = [0, 1, 5, 64, 65, 100, 190]
    pages = 12
    cache = Cache4(4, pages, heads, P, D)
    table = table_for(rng, lengths, P, pages)
    held = np.zeros((pages, P), dtype=bool)
    for r, n in enumerate(lengths):
        for t in range(n):
            held[table[r, t // P], t % P] = True
    for s in cache.scales:
        s[np.broadcast_to(~held[:, None, :, None], s.shape)] = 0x7f
        s[..., 3][~np.broadcast_to(held[:, None], s.shape[:3])] = 0xff
    block = D // 16 - 1
    if G > 1:
        cache.scales[1][table[5, 1], :, 99 - P, block] = 0x7f  # the last token of request 5: one block
        cache.scales[0][table[4, 1], :, 64 - P, 1] = 0xff      # a key: its whole rows
    q = queries(rng, len(lengths) * G, heads * g, D)
    ref = cache.attend(q, table, lengths, G)
    if G > 1:
        nan = np.isnan(ref[0])
        assert nan[5 * G + G - 1, :, 16 * block:].all() and nan[5 * G + G - 1].sum() == 16 * heads * g
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
    """Any order, duplicates, pages past the row's end, -1, empty lists, counts below and beyond the width."""
    rng = np.random.default_rng(11)
    lengths = [700, 1, 0, 333, P, 3 * P + 1]
    heads, K = 2, 9
    pages = sum(-(-n // P) for n in lengths) + 1
    cache = Cache4(5, pages, heads, P, D)
    table = table_for(rng, lengths, P, pages)
    B = len(lengths) * G
    lists = rng.integers(-2, max(lengths) // P + 3, (B, heads, K))
    lists[0, 0] = 0                     # one page nine times
    counts = rng.integers(0, K + 1, (B, heads))
    counts[0, 0], counts[-1, 0], counts[-1, 1] = K + 5, -3, 0
    q = queries(rng, B, heads * g, D)
    check_decode(*run(cuda, cache, q, table, lengths, G, lists, counts), cache.attend(q, table, lengths, G, lists, counts))
    check_decode(*run(cuda, cache, q, table, lengths, G, lists), cache.attend(q, table, lengths, G, lists), "no counts")
    out, lse = run(cuda, cache, q, table, lengths, G, lists[:, :, :0])
    assert (out == 0).all() and np.isneginf(lse.cpu().numpy()).all()


def test_exponents_scales_and_query_sizes_over_their_ranges(cuda):
    """Heads from 2^-90 to 2^60, block scales from 2^-9 to 448 in one row, rows of queries of very different
    size, a zero query, a negative softmax scale."""
    rng = np.random.default_rng(13)
    P, D, lengths = 32, 128, [150, 150, 150]
    cache = Cache4(7, 18, 4, P, D)
    cache.exps = [np.array([-90, 0, 60, 3]), np.array([60, -90, 0, -300])]
    table = table_for(rng, lengths, P, 18)
    for s in cache.scales:
        s[:, 1] = rng.integers(1, 0x7f, s[:, 1].shape)
    q = queries(rng, 3, 8, D)
    q[:, 0:2] = opaged.bf16_round(q[:, 0:2] * 2.0 ** 88)
    q[:, 2:4] = opaged.bf16_round(q[:, 2:4] * 2.0 ** -8)
    q[:, 4:6] = opaged.bf16_round(q[:, 4:6] * 2.0 ** -61)
    q[1, 6] = 0.0
    q[2, 7, ::2] = opaged.bf16_round(q[2, 7, ::2] * 2.0 ** -20)
    for sm in (D ** -0.5, -0.07):
        check_decode(*run(cuda, cache, q, table, lengths, sm_scale=sm), cache.attend(q, table, lengths, sm_scale=sm))


def test_more_requests_than_one_launch_takes(cuda):
    rng = np.random.default_rng(14)
    P, D = 16, 64
    lengths = rng.integers(0, 40, 2100)
    pages = int(sum(-(-n // P) for n in lengths)) + 1
    cache = Cache4(8, pages, 1, P, D)
    table = table_for(rng, lengths, P, pages)
    q = queries(rng, len(lengths), 2, D)
    check_decode(*run(cuda, cache, q, table, lengths), cache.attend(q, table, lengths))


def test_table_entries_outside_the_pool_read_nothing_and_lengths_are_clamped(cuda):
    rng = np.random.default_rng(15)
    P, D, lengths = 32, 128, [100, 60]
    cache = Cache4(9, 8, 2, P, D)
    for s in cache.scales:
        s[rng.permutation(8)[:2]] = 0x7f  # NaN in pages that are not read
    table = np.array([[0, -5, 1, 8], [2 ** 31 - 1, 2, 0, 0]])
    for p in (0, 1, 2):
        for s in cache.scales:
            s[p][s[p] == 0x7f] = 0x30
    q = queries(rng, 2, 4, D)
    check_decode(*run(cuda, cache, q, table, lengths), cache.attend(q, table, lengths))
    check_decode(*run(cuda, cache, q, table, [5000, -7]), cache.attend(q, table, [128, 0]))


def test_strided_queries_and_table_rows(cuda):
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(17)
    P, D, heads, g, lengths = 32, 128, 2, 3, [90, 33, 0, 1]
    cache = Cache4(11, 12, heads, P, D)
    table = table_for(rng, lengths, P, 12)
    q = queries(rng, 4, heads * g, D)
    fused = torch.full((4, (heads * g + 4) * D), float("nan"), dtype=torch.bfloat16, device=cuda)
    fused[:, 2 * D:(2 + heads * g) * D] = bf16(q, cuda).flatten(1)
    wide = torch.full((4, table.shape[1] + 3), -1, dtype=torch.int32, device=cuda)
    wide[:, :table.shape[1]] = i32(table, cuda)
    out, lse = binding.paged4_decode(
        fused[:, 2 * D:(2 + heads * g) * D].view(4, heads * g, D), cache.to(cuda),
        wide[:, :table.shape[1]], i32(lengths, cuda), D ** -0.5)
    check_decode(out, lse, cache.attend(q, table, lengths))


def test_a_pool_past_32_bit_offsets(cuda):
    """Pages whose codes and scales lie beyond 2^32 bytes in each side of the pool."""
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(18)
    P, D, heads = 64, 128, 8
    pages = 2 ** 32 // (P * D // 16 * heads) + 200
    small = Cache4(12, 40, heads, P, D)
    where = np.concatenate([np.arange(20), pages - 1 - np.arange(20)])
    at = torch.from_numpy(where).to(cuda)
    pools = [torch.empty((pages, heads, P, D // 2), dtype=torch.uint8, device=cuda) for _ in "kv"]
    scales = [torch.full((pages, heads, P, D // 16), 0x7f, dtype=torch.uint8, device=cuda) for _ in "kv"]
    for side in (0, 1):
        pools[side][at] = torch.from_numpy(small.codes[side]).to(cuda)
        scales[side][at] = torch.from_numpy(small.scales[side]).to(cuda)
    lengths = [1200, 1100]
    table = table_for(rng, lengths, P, 40)
    q = queries(rng, 2, heads * 4, D)
    used = table < 40
    far = np.where(used, where[np.where(used, table, 0)], -1)
    cache = binding.PagedCache4(*pools, *scales, *(i32(e, cuda) for e in small.exps))
    out, lse = binding.paged4_decode(bf16(q, cuda), cache, i32(far, cuda), i32(lengths, cuda), D ** -0.5)
    check_decode(out, lse, small.attend(q, table, lengths))


def test_another_stream_and_graphs_that_share_a_workspace_give_the_same_bits(cuda):
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(19)
    P, D, lengths = 64, 128, [3000, 17, 0]
    cache = Cache4(13, 60, 2, P, D)
    table = table_for(rng, [3000, 17, 100], P, 60)
    q = queries(rng, 3, 8, D)
    c, tq, tt, tl = cache.to(cuda), bf16(q, cuda), i32(table, cuda), i32(lengths, cuda)
    ws = torch.zeros(binding.paged4_workspace_bytes(c), dtype=torch.uint8, device=cuda)
    out, lse = binding.paged4_decode(tq, c, tt, tl, D ** -0.5, workspace=ws)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out2, lse2 = torch.zeros_like(out), torch.zeros_like(lse)
    with torch.cuda.stream(side):
        binding.paged4_decode(tq, c, tt, tl, D ** -0.5, workspace=ws, out=out2, lse=lse2)
    side.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    graphs, outs = [], []
    for _ in range(2):  # replayed one after the other, as the workspace asks
        graphs.append(torch.cuda.CUDAGraph())
        outs.append((torch.zeros_like(out), torch.zeros_like(lse)))
        with torch.cuda.graph(graphs[-1]):
            binding.paged4_decode(tq, c, tt, tl, D ** -0.5, workspace=ws, out=outs[-1][0], lse=outs[-1][1])
    tl[2] = 100  # a replay goes by what the buffers hold then
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    for o in outs:
        check_decode(*o, cache.attend(q, table, [3000, 17, 100]))


def test_nothing_to_do_and_refusals(cuda):
    import torch
    from sparse_mla_decode_gb300 import binding
    c = Cache4(14, 4, 2, 32, 128).to(cuda)
    none = binding.paged4_decode(torch.empty((0, 4, 128), dtype=torch.bfloat16, device=cuda), c,
                                 torch.empty((0, 2), dtype=torch.int32, device=cuda),
                                 torch.empty(0, dtype=torch.int32, device=cuda), 0.1)
    assert none[0].shape == (0, 4, 128)
    q, t, n = bf16(np.zeros((2, 4, 128)), cuda), i32([[0, 1], [2, 3]], cuda), i32([3, 4], cuda)
    ws = torch.empty(binding.paged4_workspace_bytes(c), dtype=torch.uint8, device=cuda)

    def status(**kw):
        with pytest.raises(binding.SmdError) as e:
            binding.paged4_decode(kw.get("q", q), c, t, n, 0.1, row_group=kw.get("G", 1), workspace=kw.get("ws", ws))
        return e.value.status

    assert status(ws=ws[:-16]) == binding.SMD_ERR_WORKSPACE
    assert status(ws=ws[4:]) == binding.SMD_ERR_WORKSPACE
    assert status(q=bf16(np.zeros((2, 3, 128)), cuda)) == binding.SMD_ERR_SHAPE  # 3 heads over 2
    assert status(q=bf16(np.zeros((18, 4, 128)), cuda), G=9) == binding.SMD_ERR_SHAPE
    for kw in (dict(q=q[:1]), dict(q=q.float()), dict(block_counts=n)):
        with pytest.raises(ValueError):
            binding.paged4_decode(kw.pop("q", q), c, t, n, 0.1, **kw)
    with pytest.raises(AttributeError):
        binding.paged4_decode(q, None, t, n, 0.1)


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
    cache = Cache4(6, 80, 2, P, D)
    table = rng.integers(0, 80, (len(lengths), -(-200000 // P)))  # a range of 9 tiles or more for a warp
    q = queries(rng, len(lengths) * G, 2 * g, D)
    ref = cache.attend(q, table, lengths, G)
    c = cache.to(cuda)
    args = (bf16(q, cuda), c, i32(table, cuda), i32(lengths, cuda), D ** -0.5)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    ws = torch.zeros(binding.paged4_workspace_bytes(c), dtype=torch.uint8, device=cuda)
    for with_status in (status, None):
        out, lse = binding.paged4_decode(*args, row_group=G, status=with_status, workspace=ws,
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
    check_decode(*binding.paged4_decode(*args, row_group=G, workspace=ws), ref, "after a wait that ran out")


@pytest.mark.parametrize("D,P,G,n", [(64, 16, 2, 49), (64, 48, 3, 146), (128, 16, 4, 18), (128, 64, 8, 70), (256, 16, 2, 17)])
def test_a_page_that_only_a_later_verify_row_sees_does_not_matter(cuda, D, P, G, n):
    """The bits of the rows before it are the same whatever the page holds."""
    import torch
    rng = np.random.default_rng(D + P + n)
    cache = Cache4(20, 12, 2, P, D)
    table = table_for(rng, [n], P, 12)
    q = queries(rng, G, 2 * 3, D)
    got = run(cuda, cache, q, table, [n], G)
    last, first = table[0, (n - 1) // P], (n - 1) // P * P  # the last page's tokens
    sees = [i for i in range(G) if n - G + 1 + i > first]
    before = [i for i in range(G) if i not in sees]
    assert before and sees
    cache.scales[0][last], cache.scales[1][last] = 0x7f, 0x7e
    cache.codes[1][last] = 0x77
    other = run(cuda, cache, q, table, [n], G)
    for a, b in zip(got, other):
        assert torch.equal(a[before], b[before])


@pytest.mark.parametrize("D,P,G", [(64, 16, 1), (64, 32, 2), (128, 64, 1), (256, 16, 1)])
def test_requests_of_nearly_2_to_the_31_tokens(cuda, D, P, G):
    """A length past 2^31 - P over a table that names pages of zeros beyond its first and last ones."""
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(D + P)
    W = (2 ** 31 - 1) // P
    cache = Cache4(21, 4, 1, P, D)
    q = queries(rng, G, 2, D)
    table = torch.full((1, W), 0, dtype=torch.int32, device=cuda)
    lists = np.array([[[W - 1, 3, W - 2]]] * G)
    table[0, W - 2:] = torch.tensor([2, 1], dtype=torch.int32, device=cuda)
    table[0, 3] = 3
    n = W * P - 5
    c = cache.to(cuda)
    out, lse = binding.paged4_decode(bf16(q, cuda), c, table, i32([n], cuda), D ** -0.5, row_group=G,
                                     block_lists=i32(lists, cuda))
    torch.cuda.synchronize()
    # The same tokens as a request of three pages, the last of them first in the list.
    small = np.array([[3, 2, 1]])
    ref = cache.attend(q, small, [3 * P - 5], G, np.array([[[2, 0, 1]]] * G))
    check_decode(out, lse, ref)
