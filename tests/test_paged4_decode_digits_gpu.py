"""smd_paged4_decode at 128 columns: the digits that it takes its queries as, with logits that show them.

A column far above the others takes bits from those (smd.h says how many), and its own products would drown what is left
of them. Here the keys are 0 in that column, so the logits are of the other columns alone. The oracle gets the
queries as the digits hold them, to the nearest multiple of 2^-15 of the power of two below their block's largest value (of
2^-14 of the row's where that is more), and the ordinary tolerances hold, which are small beside the values:
a digit, a scale of a set or a block's power that is wrong shows."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import paged as opaged
from oracle import paged4 as opaged4
from paged4_common import Cache4
from paged_common import check_decode, table_for, tolerances
from test_paged4_decode_gpu import queries, run

pytestmark = pytest.mark.gpu
D = 128
LENGTHS = [0, 1, 3, 128, 129, 300, 700]


def as_digits(q):
    """Queries to the nearest value that six digits in base 8 hold (ties to even)."""
    B, Hq, _ = q.shape
    x = q.reshape(B, Hq, D // 16, 16)

    def power(a):  # the exponent of the largest value; zeros have bf16's least
        return np.where(a > 0, np.frexp(a)[1] - 1, -126)
    block, row = power(np.abs(x).max(-1)), power(np.abs(q).max(-1))
    unit = np.exp2(np.maximum(block, row[..., None] - 14) - 15.0)[..., None]
    return (np.rint(x / unit) * unit).reshape(q.shape)


def check(cuda, cache, q, table, lengths, G=1, sm_scale=D ** -0.5):
    held = as_digits(q)
    want = ref, lse, reach, spread = cache.attend(held, table, lengths, G, sm_scale=sm_scale)
    t_out, t_lse = tolerances(ref, reach, spread, lse)
    seen = np.isfinite(lse)
    assert (t_out[seen] <= 0.02 * spread.max()).all() and (t_lse[seen] <= 0.01).all()
    check_decode(*run(cuda, cache, q, table, lengths, G, sm_scale=sm_scale), want)
    return held


def quiet_column(cache, head, c):
    """The keys' codes of a column become 0."""
    cache.codes[0][:, head, :, c // 2] &= 0xf0 if c % 2 == 0 else 0x0f


@pytest.mark.parametrize("g,G,P,layout", [
    (1, 1, 16, "heads"), (8, 1, 64, "tokens"), (13, 1, 64, "heads"), (16, 1, 128, "paired"), (8, 2, 256, "tokens"),
    (31, 1, 64, "heads"), (8, 4, 48, "heads"), (33, 1, 32, "heads"), (6, 8, 64, "tokens"), (64, 1, 128, "heads")])
@pytest.mark.parametrize("c", [0, 5, 16, 47, 81, 127])
def test_what_a_large_column_leaves_of_the_others(cuda, g, G, P, layout, c):
    rng = np.random.default_rng(g + G + P + c)
    pages = sum(-(-n // P) for n in LENGTHS) + 2
    cache = Cache4(g, pages, 2, P, D, layout)
    for head in range(2):
        quiet_column(cache, head, c)
    q = queries(rng, len(LENGTHS) * G, 2 * g, D)
    flat = q.reshape(-1, D)
    for row in range(len(flat)):  # by up to 2^26: its own block loses the most, the others from 2^6 or so on
        flat[row, c] = rng.choice([-1.0, 1.0]) * rng.uniform(1, 2) * 2.0 ** (row % 27)
    q = opaged.bf16_round(flat).reshape(q.shape)
    table = table_for(rng, LENGTHS, P, pages)
    held = check(cuda, cache, q, table, LENGTHS, G)
    check(cuda, cache, q, table, LENGTHS, G, sm_scale=-1.5 * D ** -0.5)
    lost = held != q
    assert lost.any() and not lost.all()


@pytest.mark.parametrize("g", [3, 8, 12, 16, 32])
def test_blocks_of_many_sizes(cuda, g):
    """Blocks down to 2^-9 of the others, where keys are as much larger, so that all of them weigh; beside a block
    up to 2^12 above them, where keys are 0."""
    rng = np.random.default_rng(g)
    P, pages = 64, sum(-(-n // 64) for n in LENGTHS) + 1
    cache = Cache4(2, pages, 1, P, D, exps=False)
    down = np.array([0, 9, 4, 7, 2, 8, 1, 6])
    k = rng.standard_normal((pages * P, 1, D // 16, 16)) * np.exp2(down - 5.0)[:, None]
    codes, scales = opaged4.quantise(opaged.bf16_round(k.reshape(-1, 1, D)), np.zeros(1))
    cache.codes[0] = np.ascontiguousarray(codes.reshape(pages, P, 1, D // 2).swapaxes(1, 2))
    cache.scales[0] = np.ascontiguousarray(scales.reshape(pages, P, 1, D // 16).swapaxes(1, 2))
    more = rng.integers(0, 13, (len(LENGTHS), g, 1, 1))
    cache.codes[0][:, :, :, :8] = 0
    q = rng.standard_normal((len(LENGTHS), g, D // 16, 16)) * np.exp2(4.0 - down)[:, None]
    q[:, :, :1] *= np.exp2(more)
    q = opaged.bf16_round(q.reshape(len(LENGTHS), g, D))
    table = table_for(rng, LENGTHS, P, pages)
    check(cuda, cache, q, table, LENGTHS)


@pytest.mark.parametrize("g", [7, 16, 29])
def test_every_digit_of_one_column(cuda, g):
    """Rows with one value that the keys see, of every mantissa, and beside it a quiet one that puts the value's last
    place at each of the digits."""
    rng = np.random.default_rng(g)
    P = 64
    lengths = [130] * 16
    pages = 3 * len(lengths) + 1
    cache = Cache4(6, pages, 1, P, D, exps=False)
    seen, quiet = 70, 66  # of one block
    for c in range(D):
        if c != seen:
            quiet_column(cache, 0, c)
    q = np.zeros((len(lengths), g, D))
    i = np.arange(len(lengths) * g)
    q[..., seen] = ((1 + i * 5 % 128 / 128) * (1 - 2 * (i % 2))).reshape(len(lengths), g)
    q[..., quiet] = np.exp2(i % 17).reshape(len(lengths), g)
    table = table_for(rng, lengths, P, pages)
    check(cuda, cache, opaged.bf16_round(q), table, lengths, sm_scale=0.5)
