"""A speculative step over the 4-bit cache, all calls together as paged_step.PagedStep makes them: tables,
norm and rotation, append, page scores and select, attention, verification, trim; against the
oracle fed with the same tokens."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import paged as opaged
from oracle import paged4 as opaged4
from paged_common import bf16, check_decode, i32
from test_verify_gpu import distributions, drawn, f32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages", [None, 5])
def test_steps_against_the_oracle(cuda, pages):
    import torch
    from sparse_mla_decode_gb300 import binding
    from sparse_mla_decode_gb300.paged_step import PagedStep
    rng = np.random.default_rng(1)
    R, P, D, heads, q_heads, width, pool, G, V = 5, 16, 64, 2, 6, 12, 60, 4, 700
    s = PagedStep(R, width, pool, q_heads, heads, D, P, pages=pages, device=cuda, bits=4)
    pools = [np.zeros((pool, heads, P, D // 2), dtype=np.uint8) for _ in "kv"]
    scales = [np.zeros((pool, heads, P, D // 16), dtype=np.uint8) for _ in "kv"]
    bounds = np.zeros((pool, heads, 2, D))
    table = np.zeros((R, width), dtype=np.int32)
    ring, state, lengths = np.arange(pool, dtype=np.int32), np.array([0, pool]), np.zeros(R, dtype=np.int32)
    freqs = np.exp2(-np.arange(16) / 2.0).astype(np.float32)[None]
    weight = opaged.bf16_round(rng.uniform(0.5, 1.5, D))
    grants = [[100, 4, 40, 4, 16], [G] * R, [G, -1, G, 50, G], [G, 30, G, G, -1], [G] * R, [G] * R]
    for step, new in enumerate(grants):
        T = 180
        _, slots, positions = s.grant(i32(new, cuda), T)
        lengths, state, _, want_slots, want_pos, table, ring, refused = opaged.block_tables(
            lengths, np.array(new), table, ring, state, P, T)
        assert not refused and np.array_equal(slots.cpu().numpy(), want_slots), step
        x = opaged.bf16_round(rng.standard_normal((T, heads, D)) * 3)
        v = opaged.bf16_round(rng.standard_normal((T, heads, D)))
        _, k = binding.qk_norm_rope(bf16(x, cuda), bf16(x, cuda), positions, f32(freqs[0], cuda), None, bf16(weight, cuda))
        k64, reach = opaged4.qk_norm_rope(x, weight, 1e-6, np.array(want_pos)[None], freqs, False)
        k = k.float().cpu().numpy().astype(np.float64)
        live = want_slots >= 0
        assert (np.abs(k - k64)[live] <= 2.0 ** -8 * np.abs(k64)[live] + 2.0 ** -18 * reach[live]).all()
        s.write(bf16(k, cuda), bf16(v, cuda), slots)
        opaged4.paged4_append(pools, scales, [None, None], bounds, [k, v], want_slots)
        assert np.array_equal(s.cache.bounds.float().cpu().numpy(), bounds)
        q = opaged.bf16_round(rng.standard_normal((R * G, q_heads, D)))
        tq = bf16(q, cuda)
        lists = counts = None
        if pages is not None:
            sc = binding.block_scores(tq, s.cache, s.table, s.lengths[s.now], row_group=G, keep_first=1, keep_last=2)
            flat = torch.full((R * G * heads, sc.stride(1)), float("nan"), dtype=torch.bfloat16, device=cuda)
            flat[:, :width] = sc.flatten(0, 1)
            idx, cnt = binding.topk_select(flat, pages)
            lists = idx.view(R * G, heads, pages).cpu().numpy()
            counts = cnt.view(R * G, heads).cpu().numpy()
        out, lse = s.attend(tq, row_group=G)
        torch.cuda.synchronize()
        assert int(s.status.item()) == 0
        vals = [opaged4.values(p, sc) for p, sc in zip(pools, scales)]
        check_decode(out, lse, opaged4.attend(q, *vals, table, lengths, D ** -0.5, G, lists, counts), f"step {step}")
        if step == 0:
            continue
        # The last G - 1 tokens of every request were drafts.
        p, dq = distributions(rng, R, G, V)
        d = drawn(rng, dq)
        u, w = rng.random((R, G - 1)), rng.random(R)
        got, accepted = s.keep(f32(p, cuda), i32(d, cuda), f32(u, cuda), f32(w, cuda), f32(dq, cuda))
        want = opaged4.verify_drafts(p, dq, d, u.astype(np.float32), w.astype(np.float32))
        assert np.array_equal(got.cpu().numpy(), want[0]) and np.array_equal(accepted.cpu().numpy(), want[1])
        lengths, state, ring = opaged4.block_trim(lengths, want[2], table, ring, state, P)
    assert np.array_equal(s.lengths[s.now].cpu().numpy(), lengths)
    assert np.array_equal(s.state[s.now].cpu().numpy(), state) and np.array_equal(s.ring.cpu().numpy(), ring)


@pytest.mark.parametrize("more", [["--bits", "4"], ["--bits", "4", "--drafts", "3"], ["--drafts", "2"]])
def test_the_command_runs(cuda, capsys, more):
    from sparse_mla_decode_gb300 import paged_step
    assert paged_step.main(["--requests", "3", "--context", "700", "--steps", "4", "--pages", "4", *more]) == 0
    assert "step over all tokens" in capsys.readouterr().out
