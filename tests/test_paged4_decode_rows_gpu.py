"""smd_paged4_decode at 128 columns over its query rows: queries of every size and shape, block
scales of either sign, values that are no numbers.

The kernel takes a block of 16 of a query's columns as six digits in base 8: exact for values of 2^-8
of the block's largest and more (bf16 has 8 bits), and off by at most 2^-16 of the block's largest, or of
2^-14 of the row's where that is more, for smaller ones. What that makes of a logit is added to
the tolerance here; paged_common.tolerances has the rest."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import paged as opaged
from paged4_common import Cache4
from paged_common import check_decode, table_for
from test_paged4_decode_gpu import queries, run

pytestmark = pytest.mark.gpu
D = 128
LENGTHS = [0, 1, 3, 128, 129, 300, 700]


def digits_reach(cache, q, sm_scale):
    """What the rounding of the queries adds to a logit, over the 2^-17 that `reach` counts with."""
    B, Hq, _ = q.shape
    blocks = np.abs(q).reshape(B, Hq, D // 16, 16)
    most = np.maximum(blocks.max(-1), 2.0 ** -14 * np.abs(q).max(-1)[..., None])[..., None]
    off = np.where(blocks >= 2.0 ** -8 * most, 0.0, 2.0 ** -16 * most).reshape(B, Hq, D)
    k = np.nanmax(np.abs(cache.values(0)), (0, 2))  # [heads, D]
    g = Hq // k.shape[0]
    return 2.0 ** 17 * abs(sm_scale) * (off * np.repeat(k, g, 0)).sum(-1)


def check(cuda, cache, q, table, lengths, G=1, sm_scale=D ** -0.5):
    ref, lse, reach, spread = cache.attend(q, table, lengths, G, sm_scale=sm_scale)
    got = run(cuda, cache, q, table, lengths, G, sm_scale=sm_scale)
    # Where logits may be off by 100 (2^17 reach) and more, e to that is no number any more; a tighter limit is.
    reach = np.minimum(reach + digits_reach(cache, q, sm_scale), 100 * 2.0 ** 17)
    check_decode(*got, (ref, lse, reach, spread))


@pytest.mark.parametrize("g,G,P,layout", [
    (1, 1, 16, "heads"), (7, 1, 64, "tokens"), (8, 1, 128, "heads"), (3, 3, 32, "heads"), (15, 1, 64, "heads"),
    (16, 1, 16, "paired"), (8, 2, 256, "tokens"), (17, 1, 64, "heads"), (31, 1, 128, "heads"), (32, 1, 48, "heads"),
    (8, 4, 64, "heads"), (33, 1, 64, "heads"), (6, 8, 64, "tokens"), (64, 1, 128, "heads")])
def test_a_column_far_above_the_others(cuda, g, G, P, layout):
    rng = np.random.default_rng(g + G + P)
    pages = sum(-(-n // P) for n in LENGTHS) + 2
    cache = Cache4(g, pages, 2, P, D, layout)
    q = queries(rng, len(LENGTHS) * G, 2 * g, D)
    flat = q.reshape(-1, D)
    for row in range(0, len(flat), 2):  # a row's, or a block's, by up to 2^25
        c = rng.integers(0, D)
        flat[row, c] *= 2.0 ** (row // 2 % 26)
        if row % 4 == 2:
            flat[row, c - c % 16:c - c % 16 + 16] *= 2.0 ** -(row // 4 % 20)
    q = opaged.bf16_round(flat).reshape(q.shape)
    check(cuda, cache, q, table_for(rng, LENGTHS, P, pages), LENGTHS, G)


@pytest.mark.parametrize("g", [4, 12, 30])
@pytest.mark.parametrize("size", [-132, -118, -60, 30, 80, 124])
def test_queries_from_the_smallest_to_the_largest(cuda, g, size):
    """The softmax scale makes up for it; rows of zeros are among them."""
    rng = np.random.default_rng(size + 200)
    P, pages = 64, sum(-(-n // 64) for n in LENGTHS) + 1
    cache = Cache4(3, pages, 1, P, D, exps=False)
    q = opaged.bf16_round(queries(rng, len(LENGTHS), g, D) * 2.0 ** size)
    q[:, 1] = 0
    q[3, :, 5:] = 0
    sm_scale = float(np.float32(D ** -0.5 * 2.0 ** -min(max(size, -100), 120)))
    check(cuda, cache, q, table_for(rng, LENGTHS, P, pages), LENGTHS, sm_scale=sm_scale)
    check(cuda, cache, q, table_for(rng, LENGTHS, P, pages), LENGTHS, sm_scale=-sm_scale)


@pytest.mark.parametrize("g,G", [(5, 1), (8, 2), (29, 1)])
def test_block_scales_of_either_sign(cuda, g, G):
    rng = np.random.default_rng(g)
    P, pages = 64, sum(-(-n // 64) for n in LENGTHS) + 1
    cache = Cache4(4, pages, 2, P, D)
    for s in cache.scales:
        s[rng.random(s.shape) < 0.3] |= 0x80
    cache.scales[0][:, :, ::7, 3] = 0x80  # and a zero with a sign
    table = table_for(rng, LENGTHS, P, pages)
    check(cuda, cache, queries(rng, len(LENGTHS) * G, 2 * g, D), table, LENGTHS, G)


@pytest.mark.parametrize("g", [2, 11, 32, 40])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_queries_that_are_no_numbers(cuda, g, bad):
    """All of such a row's outputs are NaN if it sees a token, and no other row's are."""
    rng = np.random.default_rng(g)
    P, pages = 64, sum(-(-n // 64) for n in LENGTHS) + 1
    cache = Cache4(5, pages, 1, P, D)
    table = table_for(rng, LENGTHS, P, pages)
    q = queries(rng, len(LENGTHS), g, D)
    want = cache.attend(q, table, LENGTHS)
    q[:, g // 2, 77] = bad
    out, lse = (x.float().cpu().numpy() for x in run(cuda, cache, q, table, LENGTHS))
    row = np.zeros((len(LENGTHS), g), dtype=bool)
    row[np.array(LENGTHS) > 0, g // 2] = True
    assert np.array_equal(np.isnan(lse), row) and np.array_equal(np.isnan(out).any(-1), row)
    assert np.isnan(out[row]).all()
    assert (out[np.array(LENGTHS) == 0] == 0).all()
    assert np.allclose(out[~row], want[0][~row], rtol=0.02, atol=0.02)  # the values themselves are checked above


@pytest.mark.parametrize("g", [8, 16, 32])
def test_a_nan_scale_of_k_reaches_the_rows_that_see_it(cuda, g):
    rng = np.random.default_rng(g)
    P, G, lengths = 64, 2, [200, 333, 64]
    pages = sum(-(-n // P) for n in lengths)
    cache = Cache4(6, pages, 1, P, D)
    table = table_for(rng, lengths, P, pages)
    last = [(int(table[r, (n - 1) // P]), (n - 1) % P) for r, n in enumerate(lengths)]
    p, t = last[0]
    cache.scales[0][p, 0, t, 2] = 0x7f  # the last token of request 0: its last row only
    p, t = last[1]
    cache.scales[0][p, 0, t, 7] = 0xff
    q = queries(rng, len(lengths) * G, g, D)
    ref, lse, reach, spread = cache.attend(q, table, lengths, G)
    assert np.isnan(ref[[1, 3]]).all() and not np.isnan(ref[[0, 2, 4, 5]]).any()
    out, glse = run(cuda, cache, q, table, lengths, G)
    bad = np.zeros(6, dtype=bool)
    bad[[1, 3]] = True
    assert np.isnan(out.float().cpu().numpy()[bad]).all() and np.isnan(glse.cpu().numpy()[bad]).all()
    check_decode(out[~bad], glse[~bad], (ref[~bad], lse[~bad], reach[~bad] + 1e-3, spread[~bad]))
