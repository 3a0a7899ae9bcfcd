"""smd_block_tables on the GPU: every output equals the oracle's, which goes
through the requests one by one."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import paged as opaged
from paged_common import i32, in_a_fresh_process

pytestmark = pytest.mark.gpu


def make(rng, R, P, W, spare, lo=0, hi=None):
    hi = W * P // 2 if hi is None else hi
    lengths = rng.integers(lo, hi + 1, R).astype(np.int32)
    need = -(-lengths.astype(np.int64) // P)
    pages = int(need.sum()) + spare + 1
    perm = rng.permutation(pages)
    table = rng.integers(-9, 0, (R, W)).astype(np.int32)
    at = 0
    for r in range(R):
        table[r, :need[r]] = perm[at:at + need[r]]
        at += int(need[r])
    free = perm[at:]
    taken = int(rng.integers(0, 5 * pages)) + (2 ** 40 if R % 2 else 0)
    ring = np.full(pages, -5, dtype=np.int32)
    for i, p in enumerate(free):
        ring[(taken + i) % pages] = p
    return lengths, table, ring, np.array([taken, taken + len(free)], dtype=np.int64)


def check(cuda, lengths, new, table, ring, state, P, T, stride=0):
    import torch
    from sparse_mla_decode_gb300 import binding
    R, W = table.shape
    want = opaged.block_tables(lengths, new, table, ring, state, P, T)
    wide = torch.full((R, W + stride), -77, dtype=torch.int32, device=cuda)
    wide[:, :W] = i32(table, cuda)
    tring = i32(ring, cuda)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    got = binding.block_tables(i32(lengths, cuda), i32(new, cuda), wide[:, :W], tring,
                               torch.from_numpy(state).to(cuda), P, T, status=status)
    torch.cuda.synchronize()
    names = ("new_lengths", "new_state", "starts", "slots", "positions")
    for name, g, w in zip(names, got, want):
        assert np.array_equal(g.cpu().numpy().astype(np.int64), np.asarray(w, dtype=np.int64)), name
    assert np.array_equal(wide[:, :W].cpu().numpy(), want[5]), "table"
    assert (wide[:, W:] == -77).all()
    assert np.array_equal(tring.cpu().numpy(), want[6]), "ring"
    assert int(status.item()) == (binding.SMD_ERR_PAGES if want[7] else 0)
    return want


@pytest.mark.parametrize("R,P,W,new,spare", [
    (1, 16, 4, 1, 10), (7, 64, 9, 3, 20), (300, 16, 40, 1, 400), (513, 32, 12, 40, 3000),
    (1025, 1, 20, 4, 9000), (8192, 16, 3, 9, 9000), (5, 7, 300, 800, 900), (64, 128, 600, 5000, 4000)])
def test_steps_and_prompts(cuda, R, P, W, new, spare):
    rng = np.random.default_rng(R)
    lengths, table, ring, state = make(rng, R, P, W, spare)
    n = rng.integers(0, new + 1, R).astype(np.int32)
    n[rng.random(R) < 0.2] = -1
    check(cuda, lengths, n, table, ring, state, P, int(np.maximum(n, 0).sum()) + 9, stride=3)


@pytest.mark.parametrize("seed", range(12))
def test_refusals_for_pages_width_and_slots(cuda, seed):
    rng = np.random.default_rng(seed)
    R, P, W = int(rng.integers(2, 900)), int(rng.choice([4, 16, 48])), 6
    lengths, table, ring, state = make(rng, R, P, W, int(rng.integers(0, R)), hi=W * P)
    n = rng.integers(-1, 3 * P, R).astype(np.int32)
    T = int(np.maximum(n, 0).sum() * rng.random())
    want = check(cuda, lengths, n, table, ring, state, P, T)
    assert want[7]


def test_a_request_may_fill_its_last_page_when_no_page_is_free(cuda):
    P, lengths = 16, np.array([10, 16, 5], dtype=np.int32)
    table = np.array([[0, -1], [1, -1], [2, -1]], dtype=np.int32)
    ring, state = np.array([0, 0, 0], dtype=np.int32), np.array([3, 3], dtype=np.int64)
    want = check(cuda, lengths, np.array([6, 1, 2], dtype=np.int32), table, ring, state, P, 20)
    assert list(want[0]) == [16, 16, 7] and want[7]


def test_extremes(cuda):
    """No tokens, no room, the longest request that an int holds, lengths out of range."""
    rng = np.random.default_rng(20)
    lengths, table, ring, state = make(rng, 6, 16, 8, 10)
    check(cuda, lengths, np.zeros(6, dtype=np.int32), table, ring, state, 16, 0)
    check(cuda, lengths, np.full(6, 2 ** 31 - 1, dtype=np.int32), table, ring, state, 16, 5)
    check(cuda, np.array([-5, 2 ** 31 - 1, 3, 0, 1, 2], dtype=np.int32),
          np.array([3, 1, 0, -1, -2 ** 31, 4], dtype=np.int32), table, ring, state, 16, 50)


def test_pages_go_round(cuda):
    """Steps of a serving loop: what is granted and returned stays a partition of
    the pool, and every live token keeps its slot."""
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(21)
    R, P, W, pages = 20, 16, 10, 90
    lengths = torch.zeros(R, dtype=torch.int32, device=cuda)
    table = torch.zeros((R, W), dtype=torch.int32, device=cuda)
    ring = torch.arange(pages, dtype=torch.int32, device=cuda)
    state = torch.tensor([0, pages], dtype=torch.int64, device=cuda)
    slots_of = [[] for _ in range(R)]
    for _ in range(120):
        new = rng.integers(0, 30, R) * (rng.random(R) < 0.4)
        new[rng.random(R) < 0.1] = -1
        lengths, state, starts, slots, _ = binding.block_tables(
            lengths, i32(new, cuda), table, ring, state, P, 700)
        torch.cuda.synchronize()
        st, sl = starts.cpu().numpy(), slots.cpu().numpy()
        for r in range(R):
            slots_of[r] = [] if new[r] < 0 else slots_of[r] + list(sl[st[r]:st[r + 1]])
        assert [len(x) for x in slots_of] == lengths.tolist()
        live = [s for x in slots_of for s in x]
        assert len(set(live)) == len(live)
        t = table.cpu().numpy()
        held = [t[r, j] for r in range(R) for j in range(-(-len(slots_of[r]) // P))]
        a, b = state.tolist()
        free = [int(ring[i % pages]) for i in range(a, b)]
        assert sorted(held + free) == list(range(pages))


def test_streams_and_binding_refusals(cuda):
    import torch
    from sparse_mla_decode_gb300 import binding
    n = i32([3], cuda)
    table, ring = i32([[0, 0]], cuda), i32([0, 1], cuda)
    state = torch.tensor([0, 2], dtype=torch.int64, device=cuda)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = binding.block_tables(i32([0], cuda), n, table, ring, state, 2, 4, stream=side)
    side.synchronize()
    assert got[3].tolist() == [0, 1, 2, -1]
    with pytest.raises(ValueError):
        binding.block_tables(n, n, table, ring, state, 2, 4, new_lengths=n)
    with pytest.raises(ValueError):
        binding.block_tables(n, n, table, ring, state, 2)
    with pytest.raises(ValueError):
        binding.block_tables(n.long(), n, table, ring, state, 2, 4)
    with pytest.raises(binding.SmdError) as e:
        binding.block_tables(n, n, table, ring, state, 0, 4)
    assert e.value.status == binding.SMD_ERR_SHAPE


def many_requests():
    import torch
    rng = np.random.default_rng(30)
    for R in (6063, 6064, 6100, 6143, 6144):
        lengths, table, ring, state = make(rng, R, 16, 3, 7000)
        n = rng.integers(-1, 4, R).astype(np.int32)
        check(torch.device("cuda:0"), lengths, n, table, ring, state, 16, 3 * R)


def test_requests_whose_sums_fill_48_kb_are_a_process_first_call(cuda):
    """The limit that a larger call raises is not there yet."""
    in_a_fresh_process("import test_block_tables_gpu as t; t.many_requests()")
