"""What paged_step.PagedStep.keep takes off, without a GPU: the calls that it makes are replaced by their oracles."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import paged4 as opaged4
from sparse_mla_decode_gb300 import binding
from sparse_mla_decode_gb300.paged_step import PagedStep

P = 16


class Cache:
    page_size = P


def step_of(before, now, monkeypatch, accepted, G):
    """A step whose last grant took the lengths from `before` to `now`, and what trim was asked for."""
    torch = pytest.importorskip("torch")
    s = PagedStep.__new__(PagedStep)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    s.cache, s.now = Cache(), 1
    s.lengths = [i32(before), i32(now)]
    s.state = [torch.zeros(2, dtype=torch.int64) for _ in range(2)]
    s.table = torch.arange(16 * len(now), dtype=torch.int32).view(len(now), 16)
    s.ring = torch.zeros(64, dtype=torch.int32)
    s.state[1] += 40
    ring0 = s.ring.clone()

    def verify(target, tokens, accept, sample, draft=None):
        return i32(np.zeros((len(now), G))), i32(accepted), i32([G - 1 - a for a in accepted])

    def trim(lengths, drop, table, ring, state, page_size, new_lengths=None, new_state=None):
        new, st, r = opaged4.block_trim(lengths.numpy(), drop.numpy(), table.numpy(), ring.numpy(), state.numpy(), page_size)
        new_lengths.copy_(torch.from_numpy(new))
        new_state.copy_(torch.from_numpy(st))
        ring.copy_(torch.from_numpy(r))
        return new_lengths, new_state

    monkeypatch.setattr(binding, "verify_drafts", verify)
    monkeypatch.setattr(binding, "block_trim", trim)
    target = torch.zeros(len(now), G, 8)
    s.keep(target, None, None, None)
    return s.lengths[s.now].tolist(), int(s.state[s.now][1]) - 40, ring0


@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_only_tokens_of_the_last_grant_come_off(monkeypatch, G):
    """Requests of 0 to 12 new tokens, whatever the verification says of them: of n < G the drafts are n - 1."""
    grants, before, accepted = [], [], []
    for n in [*range(0, G + 3), 12]:
        for a in range(G):
            for length in (0, 1, 15, 16, 17, 40):
                grants.append(n)
                before.append(length)
                accepted.append(a)
    now = [b + n for b, n in zip(before, grants)]
    got, back, _ = step_of(before, now, monkeypatch, accepted, G)
    want = [e - max(min(n, G) - 1 - a, 0) for e, n, a in zip(now, grants, accepted)]
    assert got == want
    assert all(x >= b for x, b in zip(got, before))
    assert back == sum(-(-e // P) - -(-w // P) for e, w in zip(now, want))


def test_ended_requests_stay_ended(monkeypatch):
    got, back, _ = step_of([50, 16, 0], [0, 0, 0], monkeypatch, [0, 2, 1], 4)
    assert got == [0, 0, 0] and back == 0
