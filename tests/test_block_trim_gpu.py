"""smd_block_trim on the GPU against a plain walk over the requests: equal."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import paged4 as opaged4
from paged_common import i32

pytestmark = pytest.mark.gpu


def check(cuda, lengths, drop, table, ring, state, P, stride=0):
    import torch
    from sparse_mla_decode_gb300 import binding
    wide = torch.full((table.shape[0], table.shape[1] + stride), -7, dtype=torch.int32, device=cuda)
    wide[:, :table.shape[1]] = i32(table, cuda)
    r = i32(ring, cuda)
    st = torch.tensor(np.asarray(state), dtype=torch.int64, device=cuda)
    got = binding.block_trim(i32(lengths, cuda), i32(drop, cuda), wide[:, :table.shape[1]], r, st, P)
    torch.cuda.synchronize()
    want = opaged4.block_trim(lengths, drop, table, ring, state, P)
    assert np.array_equal(got[0].cpu().numpy(), want[0]), "lengths"
    assert np.array_equal(got[1].cpu().numpy(), want[1]), "state"
    assert np.array_equal(r.cpu().numpy(), want[2]), "ring"
    assert np.array_equal(wide[:, :table.shape[1]].cpu().numpy(), table), "the table stays"


def pool(rng, lengths, P, W, spare):
    """A table of distinct pages, the ring of the others, and its state."""
    need = [-(-n // P) for n in lengths]
    pages = sum(need) + spare
    perm = rng.permutation(pages)
    table = np.full((len(lengths), W), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        at += n
    taken = int(rng.integers(0, 5 * pages + 1))
    ring = np.full(pages, -1, dtype=np.int32)
    ring[(taken + np.arange(spare)) % pages] = perm[at:]
    return table, ring, [taken, taken + spare]


@pytest.mark.parametrize("R,P,hi,drop,stride", [
    (1, 16, 40, 7, 0), (5, 64, 1000, 3, 2), (128, 16, 300, 300, 0), (129, 32, 100, 8, 1), (700, 16, 90, 90, 0),
    (2000, 48, 5000, 5000, 0), (8192, 16, 33, 20, 0), (1, 16, 60000, 60000, 0), (3, 256, 100000, 70000, 5)])
def test_sizes(cuda, R, P, hi, drop, stride):
    rng = np.random.default_rng(R + P)
    lengths = rng.integers(0, hi + 1, R)
    lengths[0] = hi
    table, ring, state = pool(rng, lengths, P, max(-(-hi // P), 1) + 1, 5)
    check(cuda, lengths, rng.integers(0, drop + 1, R), table, ring, state, P, stride)


def test_borders_of_pages_negative_drops_and_lengths_out_of_range(cuda):
    rng = np.random.default_rng(1)
    P, W = 16, 5
    lengths = np.array([0, 1, 15, 16, 17, 32, 33, 80, 64, 80, 16, 16])
    table, ring, state = pool(rng, lengths, P, W, 3)
    drop = np.array([5, 1, 14, 15, 1, 0, 1, 2 ** 31 - 1, -4, -2 ** 31, 16, 17])
    check(cuda, lengths, drop, table, ring, state, P)
    lengths[7], lengths[9], lengths[0] = 10 ** 9, 2 ** 31 - 1, -9  # clamped to the row, and to 0
    check(cuda, lengths, drop, table, ring, state, P)


def test_no_requests_and_none_that_give_back(cuda):
    import torch
    from sparse_mla_decode_gb300 import binding
    e = torch.empty(0, dtype=torch.int32, device=cuda)
    st = torch.tensor([3, 9], dtype=torch.int64, device=cuda)
    n, s = binding.block_trim(e, e, torch.empty((0, 2), dtype=torch.int32, device=cuda), i32(np.arange(10), cuda), st, 16)
    assert n.numel() == 0 and s.tolist() == [3, 9]
    rng = np.random.default_rng(2)
    table, ring, state = pool(rng, [20, 30], 16, 2, 4)
    check(cuda, np.array([20, 30]), np.array([3, 0]), table, ring, state, 16)


def test_a_table_that_names_more_than_the_pool_writes_the_ring_once_around(cuda):
    """Rows of a table that are no pool's: nothing is written outside the ring."""
    import torch
    from sparse_mla_decode_gb300 import binding
    table = np.arange(40).reshape(4, 10)
    mem = torch.full((24,), -3, dtype=torch.int32, device=cuda)
    st = torch.tensor([0, 5], dtype=torch.int64, device=cuda)
    _, s = binding.block_trim(i32([160] * 4, cuda), i32([160] * 4, cuda), i32(table, cuda), mem[8:16], st, 16)
    torch.cuda.synchronize()
    assert s.tolist() == [0, 45] and (mem[:8] == -3).all() and (mem[16:] == -3).all()


def test_tables_then_trim_go_round_and_in_a_graph(cuda):
    """Steps of drafted tokens of which some are taken back: no page is lost or given twice."""
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(3)
    R, P, W, pages, G = 17, 16, 8, 80, 5
    table = torch.zeros((R, W), dtype=torch.int32, device=cuda)
    ring = torch.arange(pages, dtype=torch.int32, device=cuda)
    lengths = [torch.zeros(R, dtype=torch.int32, device=cuda) for _ in "ab"]
    state = [torch.tensor([0, pages], dtype=torch.int64, device=cuda) for _ in "ab"]
    new, drop = torch.zeros(R, dtype=torch.int32, device=cuda), torch.zeros(R, dtype=torch.int32, device=cuda)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    held = dict(starts=torch.zeros(R + 1, dtype=torch.int32, device=cuda),
                slots=torch.zeros(R * G, dtype=torch.int32, device=cuda),
                positions=torch.zeros(R * G, dtype=torch.int32, device=cuda))

    def step():
        binding.block_tables(lengths[0], new, table, ring, state[0], P, new_lengths=lengths[1], new_state=state[1],
                             status=status, **held)
        binding.block_trim(lengths[1], drop, table, ring, state[1], P, new_lengths=lengths[0], new_state=state[0])

    graph = torch.cuda.CUDAGraph()
    step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    plain = np.zeros(R, dtype=int)
    for _ in range(60):
        n, d = rng.integers(0, G + 1, R), rng.integers(0, G, R)
        ended = rng.random(R) < 0.05
        n = np.where(ended, -1, np.where(plain + G > P * W, 0, n))
        new.copy_(i32(n, cuda))
        drop.copy_(i32(d, cuda))
        graph.replay()
        torch.cuda.synchronize()
        plain = np.where(ended, 0, np.maximum(plain + np.maximum(n, 0) - d, 0))
        assert np.array_equal(lengths[0].cpu().numpy(), plain) and int(status.item()) == 0
        taken, given = state[0].tolist()
        free = ring.cpu().numpy()[np.arange(taken, given) % pages]
        t = table.cpu().numpy()
        used = np.concatenate([t[r, :-(-plain[r] // P)] for r in range(R)])
        assert np.array_equal(np.sort(np.concatenate([free, used])), np.arange(pages))
