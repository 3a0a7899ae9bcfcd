"""smd_block_scores on the GPU against the 64-bit oracle. Tolerance: bf16's
half unit (2^-8 of the value) and the fp32 sum of up to 512 products, 2^-17 of
the sum of their sizes (16 columns a step, each at 2^-22, and room)."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import paged as opaged
from paged_common import Cache, bf16, i32, in_a_fresh_process, table_for

pytestmark = pytest.mark.gpu


def check(cuda, cache, q, table, lengths, G=1, keep=(0, 0), **kw):
    import torch
    from sparse_mla_decode_gb300 import binding
    got = binding.block_scores(bf16(q, cuda), kw.pop("c", None) or cache.to(cuda), i32(table, cuda),
                               i32(lengths, cuda), row_group=G, keep_first=keep[0],
                               keep_last=keep[1], **kw)
    torch.cuda.synchronize()
    want = opaged.block_scores(q, cache.bounds, table, lengths, cache.P, G, *keep)
    have = got.float().cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(have), np.isnan(want))
    assert np.array_equal(np.isinf(have), np.isinf(want))
    fin = np.isfinite(want)
    size = np.abs(q).max() * np.abs(cache.bounds).max() * cache.D
    assert (np.abs(have[fin] - want[fin]) <= 2.0 ** -8 * np.abs(want[fin]) + 2.0 ** -17 * size).all()
    return got


@pytest.mark.parametrize("D,P,heads,g,G,keep", [
    (128, 64, 2, 8, 1, (0, 0)), (128, 16, 3, 1, 4, (1, 2)), (128, 32, 1, 3, 2, (0, 1)),
    (128, 48, 2, 7, 3, (2, 0)), (128, 64, 1, 16, 8, (1, 1)), (64, 16, 2, 5, 1, (0, 0)),
    (64, 64, 1, 17, 2, (0, 0)), (64, 32, 4, 2, 5, (0, 3)), (256, 16, 1, 4, 1, (0, 0)),
    (256, 64, 2, 12, 2, (1, 1)), (128, 64, 1, 128, 4, (0, 0)), (256, 16, 1, 128, 8, (0, 0))])
def test_scores(cuda, D, P, heads, g, G, keep):
    rng = np.random.default_rng(D + P + g)
    lengths = [0, 1, P - 1, P, P + 1, 9 * P + 3, 40 * P, 150 * P - 1]
    pages = sum(-(-n // P) for n in lengths) + 2
    cache = Cache(1, pages, heads, P, D)
    table = table_for(rng, lengths, P, pages, extra=3)
    q = opaged.bf16_round(rng.standard_normal((len(lengths) * G, heads * g, D)))
    check(cuda, cache, q, table, lengths, G, keep)


def test_the_score_bounds_every_key(cuda):
    """After an append, no product with a key exceeds its page's score by more
    than the score's rounding."""
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(2)
    P, D, n = 32, 128, 300
    c = binding.PagedCache.empty(10, 1, P, D, device=cuda)
    k = opaged.bf16_round(rng.standard_normal((n, 1, D)))
    binding.paged_append(c, bf16(k, cuda), bf16(k, cuda), i32(np.arange(n), cuda))
    q = opaged.bf16_round(rng.standard_normal((1, 4, D)))
    s = binding.block_scores(bf16(q, cuda), c, i32([np.arange(10)], cuda), i32([n], cuda))
    torch.cuda.synchronize()
    s = s.float().cpu().numpy()[0, 0]
    dots = (k[:, 0] @ q[0].T).max(1)
    for j in range(10):
        assert dots[j * P:(j + 1) * P].max() <= s[j] * (1 + 2.0 ** -7), j


def test_output_strides_bad_pages_and_a_cache_of_bounds(cuda):
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(3)
    P, D, heads, lengths = 16, 64, 2, [100, 250]
    cache = Cache(2, 30, heads, P, D)
    table = table_for(rng, lengths, P, 30)
    table[0, 2], table[1, 5] = -1, 30
    q = opaged.bf16_round(rng.standard_normal((2, 6, D)))
    c = binding.PagedCache(bounds=bf16(cache.bounds, cuda), page_size=P)
    W = table.shape[1]
    wide = torch.zeros((2, heads, W + 5), dtype=torch.bfloat16, device=cuda)
    check(cuda, cache, q, table, lengths, c=c, out=wide[:, :, :W])
    assert (wide[:, :, W:] == 0).all()


def test_the_scores_go_to_the_select(cuda):
    """NaN past a row's pages: the select gives no page the row does not have,
    and the kept ones first."""
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(4)
    P, D, heads, lengths, K = 16, 128, 2, [500, 40, 0, 161], 6
    cache = Cache(3, 60, heads, P, D)
    table = table_for(rng, lengths, P, 60)
    q = opaged.bf16_round(rng.standard_normal((4, 8, D)))
    s = check(cuda, cache, q, table, lengths, keep=(1, 2))
    full = torch.empty((4 * heads, s.stride(1)), dtype=torch.bfloat16, device=cuda).fill_(float("nan"))
    full[:, :table.shape[1]] = s.flatten(0, 1)
    idx, cnt = binding.topk_select(full, K)
    torch.cuda.synchronize()
    idx, cnt = idx.view(4, heads, K).cpu().numpy(), cnt.view(4, heads).cpu().numpy()
    for b, n in enumerate(lengths):
        have = -(-n // P)
        assert (cnt[b] == min(K, have)).all()
        for h in range(heads):
            got = set(idx[b, h, :cnt[b, h]])
            assert got <= set(range(have))
            assert {j for j in (0, have - 2, have - 1) if 0 <= j < have} <= got


def test_refusals(cuda):
    import torch
    from sparse_mla_decode_gb300 import binding
    cache = Cache(4, 4, 2, 32, 128)
    c = cache.to(cuda)
    q, t, n = bf16(np.zeros((2, 4, 128)), cuda), i32([[0, 1], [2, 3]], cuda), i32([3, 4], cuda)
    bare = binding.PagedCache(c.k, c.v, c.k_scale, c.v_scale)
    for kw, code in ((dict(c=bare), binding.SMD_ERR_NULL), (dict(first=-1), binding.SMD_ERR_SHAPE),
                     (dict(q=bf16(np.zeros((2, 258, 128)), cuda)), binding.SMD_ERR_SHAPE)):
        with pytest.raises(binding.SmdError) as e:
            binding.block_scores(kw.get("q", q), kw.get("c", c), t, n, keep_first=kw.get("first", 0))
        assert e.value.status == code
    with pytest.raises(ValueError):
        binding.block_scores(q, c, t, n, out=torch.empty((2, 2, 3), dtype=torch.bfloat16, device=cuda))


# Query rows whose fragments fill 48 KB of shared memory to the byte: 24, 12 and 6 MMAs.
FULL = [(64, 1, 64, 3), (128, 2, 16, 6), (128, 1, 32, 3), (128, 1, 24, 4), (256, 1, 8, 6), (256, 1, 24, 2)]


def fill_48_kb():
    import torch
    cuda = torch.device("cuda:0")
    for D, heads, g, G in FULL:
        rng = np.random.default_rng(D + g)
        P, lengths = 32, [0, 70, 1000]
        cache = Cache(5, 40, heads, P, D)
        table = table_for(rng, lengths, P, 40)
        q = opaged.bf16_round(rng.standard_normal((len(lengths) * G, heads * g, D)))
        check(cuda, cache, q, table, lengths, G)


def test_queries_that_fill_48_kb_are_a_process_first_call(cuda):
    """The limit that a larger call raises is not there yet."""
    in_a_fresh_process("import test_block_scores_gpu as t; t.fill_48_kb()")


def test_a_request_of_nearly_2_to_the_31_tokens(cuda):
    """As long as the table allows: every page is scored, up to the last one."""
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(5)
    P, D, width = 48, 64, 2 ** 31 // 48
    cache = Cache(4, 5, 1, P, D)
    table = torch.full((1, width), -1, dtype=torch.int32, device=cuda)
    at = [0, 1, width // 2, width - 2, width - 1]
    table[0, at] = i32([3, 1, 4, 0, 2], cuda)
    q = opaged.bf16_round(rng.standard_normal((1, 3, D)))
    c = binding.PagedCache(bounds=bf16(cache.bounds, cuda), page_size=P)
    want = opaged.block_scores(q, cache.bounds, np.array([[3, 1, 4, 0, 2]]), [5 * P], P, 1)[0, 0]
    for n in (width * P, width * P - P + 1, width * P - P):  # the last page is seen whole, a token, not
        s = binding.block_scores(bf16(q, cuda), c, table, i32([n], cuda))[0, 0]
        sees = -(-n // P)
        assert bool(torch.isnan(s[sees:]).all()) and not bool(torch.isnan(s[:sees]).any())
        assert int((s[:sees] != 0).sum()) == 5 - (width - sees)
        got = s[at].float().cpu().numpy()[:5 - (width - sees)]
        size = np.abs(q).max() * np.abs(cache.bounds).max() * D
        assert (np.abs(got - want[:len(got)]) <= 2.0 ** -8 * np.abs(want[:len(got)]) + 2.0 ** -17 * size).all()
