"""paged_step.PagedStep.keep on the GPU: requests that the step granted nothing (idle, refused for pages, refused for
their row) or less than the others keep what they had."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import paged as opaged
from oracle import paged4 as opaged4
from paged_common import i32
from test_verify_gpu import distributions, drawn, f32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [4, 8])
def test_requests_that_were_granted_less_lose_nothing_older(cuda, bits):
    import torch
    from sparse_mla_decode_gb300.paged_step import PagedStep
    rng = np.random.default_rng(bits)
    R, P, D, heads, q_heads, width, pool, G, V = 8, 16, 64, 2, 4, 6, 22, 4, 300
    s = PagedStep(R, width, pool, q_heads, heads, D, P, device=cuda, bits=bits)
    table = np.zeros((R, width), dtype=np.int32)
    ring, state, lengths = np.arange(pool, dtype=np.int32), np.array([0, pool]), np.zeros(R, dtype=np.int32)

    def grant(new, T=400):
        nonlocal lengths, state, table, ring
        before = lengths.copy()
        _, slots, _ = s.grant(i32(new, cuda), T)
        lengths, state, _, want, _, table, ring, refused = opaged.block_tables(lengths, np.array(new), table, ring, state, P, T)
        assert np.array_equal(slots.cpu().numpy(), want)
        assert bool(refused) == (int(s.status.item()) != 0)
        s.status.zero_()
        return lengths - before

    def keep(accept, tokens=None):
        nonlocal lengths, state, ring
        p, dq = distributions(rng, R, G, V)
        d = drawn(rng, dq)
        if tokens is not None:
            d[tokens == -1] = -1
        accept = np.broadcast_to(np.float32(accept), (R, G - 1))
        w = rng.random(R)
        _, accepted = s.keep(f32(p, cuda), i32(d, cuda), f32(accept, cuda), f32(w, cuda), f32(dq, cuda))
        _, a, _ = opaged4.verify_drafts(p, dq, d, accept, w.astype(np.float32))
        assert np.array_equal(accepted.cpu().numpy(), a)
        drop = np.maximum(np.minimum(granted, G) - 1 - a, 0)
        lengths, state, ring = opaged4.block_trim(lengths, drop, table, ring, state, P)
        assert s.lengths[s.now].tolist() == lengths.tolist()
        assert np.array_equal(s.state[s.now].cpu().numpy(), state) and np.array_equal(s.ring.cpu().numpy(), ring)
        return a

    grant([20, 33, 16, 94, 40, 1, 17, 48])  # 94 of the 96 that a row holds; 21 pages of 22
    # idle, idle with its last page full, refused for its row, and all drafts refused
    old = lengths.copy()
    granted = grant([G, 0, 0, G, G, G, 2, 1])
    assert granted.tolist() == [G, 0, 0, 0, G, G, 2, 1]
    a = keep(1e9)
    assert (a == 0).all() and (lengths == old + np.minimum(granted, 1)).all()
    # the pool runs out: refused for pages
    old = lengths.copy()
    granted = grant([30, 0, 40, 1, G, G, G, 3])
    assert (granted == 0).sum() >= 2
    keep(1e9)
    assert (lengths >= old).all()
    # fewer drafts than the others', ended by a token outside the vocabulary, all of which stay
    old = lengths.copy()
    granted = grant([2, 3, 0, 1, G, 2, 3, 1])
    tokens = np.zeros((R, G - 1), dtype=int)
    for r, n in enumerate(granted):
        tokens[r, max(n - 1, 0):] = -1
    a = keep(0.0, tokens)
    assert (a == np.maximum(granted, 1) - 1).all() and (lengths == old + granted).all()
    # a request has ended
    granted = grant([-1, G, G, 0, -1, G, G, G])
    keep(1e9)
    assert lengths[0] == 0 and lengths[4] == 0


def test_a_step_in_a_graph(cuda):
    """Two steps captured and replayed, of which one request is idle and one cannot grow."""
    import torch
    from sparse_mla_decode_gb300.paged_step import PagedStep
    R, P, D, width, G, V = 4, 16, 64, 4, 3, 50
    s = PagedStep(R, width, R * width, 2, 1, D, P, device=cuda, bits=4)
    s.grant(i32([5, 20, 64, 30], cuda), 200)
    new = i32([G, 0, G, G], cuda)
    p = torch.full((R, G, V), 1.0 / V, device=cuda)
    d = torch.zeros((R, G - 1), dtype=torch.int32, device=cuda)
    refuse = torch.full((R, G - 1), 2.0, device=cuda)
    w = torch.full((R,), 0.5, device=cuda)

    def step():
        _, slots, _ = s.grant(new, R * G)
        return s.keep(p, d, refuse, w)
    now = s.now
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(), step()
    torch.cuda.synchronize()
    assert s.now == now and s.lengths[now].tolist() == [7, 20, 64, 32]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(), step()
    for i in range(3):
        graph.replay()
        assert s.lengths[now].tolist() == [9 + 2 * i, 20, 64, 34 + 2 * i]
    taken, given = s.state[now].tolist()
    assert taken - given + R * width == sum(-(-n // P) for n in s.lengths[now].tolist())
