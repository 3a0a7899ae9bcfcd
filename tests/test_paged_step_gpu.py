"""The paged calls together, as paged_step.PagedStep makes them: prompts,
steps with verify rows, requests that end and others that take their pages,
against the 64-bit oracle fed with the same tokens."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import paged as opaged
from paged_common import bf16, check_decode, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages", [None, 5])
def test_steps_against_the_oracle(cuda, pages):
    import torch
    from sparse_mla_decode_gb300 import binding
    from sparse_mla_decode_gb300.paged_step import PagedStep
    rng = np.random.default_rng(1)
    R, P, D, heads, q_heads, width, pool, G = 5, 16, 64, 2, 6, 12, 40, 2
    s = PagedStep(R, width, pool, q_heads, heads, D, P, pages=pages, device=cuda)
    codes = [np.zeros((pool, heads, P, D), dtype=np.uint8) for _ in "kv"]
    scales = [np.zeros((pool, heads), dtype=np.float32) for _ in "kv"]
    bounds = np.zeros((pool, heads, 2, D))
    table = np.zeros((R, width), dtype=np.int32)
    ring, state, lengths = np.arange(pool, dtype=np.int32), np.array([0, pool]), np.zeros(R, dtype=np.int32)
    grants = [[100, 3, 40, 0, 16], [2] * R, [1, -1, 2, 50, 1], [0, 30, 2, 1, -1], [2] * R]
    for step, new in enumerate(grants):
        T = 160
        _, slots, _ = s.grant(i32(new, cuda), T)
        lengths, state, _, want_slots, _, table, ring, refused = opaged.block_tables(
            lengths, np.array(new), table, ring, state, P, T)
        assert not refused and np.array_equal(slots.cpu().numpy(), want_slots), step
        x = [opaged.bf16_round(rng.standard_normal((T, heads, D)) * 2.0 ** rng.integers(-3, 3)) for _ in "kv"]
        s.write(bf16(x[0], cuda), bf16(x[1], cuda), slots)
        opaged.paged_append(codes, scales, bounds, x, want_slots)
        q = opaged.bf16_round(rng.standard_normal((R * G, q_heads, D)))
        tq = bf16(q, cuda)
        lists = counts = None
        if pages is not None:
            sc = binding.block_scores(tq, s.cache, s.table, s.lengths[s.now], row_group=G, keep_first=1,
                                      keep_last=2)
            flat = torch.full((R * G * heads, sc.stride(1)), float("nan"), dtype=torch.bfloat16, device=cuda)
            flat[:, :width] = sc.flatten(0, 1)
            idx, cnt = binding.topk_select(flat, pages)
            lists = idx.view(R * G, heads, pages).cpu().numpy()
            counts = cnt.view(R * G, heads).cpu().numpy()
        out, lse = s.attend(tq, row_group=G)
        torch.cuda.synchronize()
        assert int(s.status.item()) == 0
        ref = opaged.paged_decode(q, codes, scales, table, lengths, D ** -0.5, G, lists, counts)
        check_decode(out, lse, ref, f"step {step}")
    assert np.array_equal(s.lengths[s.now].cpu().numpy(), lengths)
    assert np.array_equal(s.state[s.now].cpu().numpy(), state)


def test_the_command_runs(cuda, capsys):
    from sparse_mla_decode_gb300 import paged_step
    assert paged_step.main(["--requests", "3", "--context", "700", "--steps", "4", "--pages", "4"]) == 0
    assert "step over all tokens" in capsys.readouterr().out


@pytest.mark.parametrize("steps", [1, 3])
def test_the_command_runs_an_odd_number_of_steps(cuda, capsys, steps):
    """The table has room for them all: the status is checked by the command."""
    from sparse_mla_decode_gb300 import paged_step
    assert paged_step.main(["--requests", "2", "--context", "64", "--steps", str(steps), "--pages", "2"]) == 0
    assert "step over all tokens" in capsys.readouterr().out
