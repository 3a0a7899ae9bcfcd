"""python -m sparse_mla_decode_gb300.paged_step --bits 4: keys and queries of one kind."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("drafts", [0, 2])
def test_the_command_norms_and_turns_all_keys_and_queries_of_a_4_bit_cache(cuda, monkeypatch, drafts):
    """What is written and what is asked with came out of the rotation, at the positions that it stands at."""
    import torch
    from sparse_mla_decode_gb300 import binding, paged_step
    turned, written, asked = [], [], []
    rope, append, decode = binding.qk_norm_rope, binding.paged4_append, binding.paged4_decode

    def spy_rope(q, k, positions, *a, **kw):
        out = rope(q, k, positions, *a, **kw)
        turned.extend((t, positions) for t in out if t is not None)
        return out

    def spy_append(cache, k, v, slots, **kw):
        written.append(k)
        return append(cache, k, v, slots, **kw)

    def spy_decode(q, cache, table, lengths, *a, **kw):
        asked.append(q)
        if not torch.cuda.is_current_stream_capturing():
            G = q.shape[0] // lengths.numel()
            want = (lengths[:, None] - G + torch.arange(G, device=cuda)).flatten().tolist()
            got = [p.flatten().tolist() for t, p in turned if t is q]
            if got:
                assert got[0] == want
        return decode(q, cache, table, lengths, *a, **kw)

    monkeypatch.setattr(binding, "qk_norm_rope", spy_rope)
    monkeypatch.setattr(binding, "paged4_append", spy_append)
    monkeypatch.setattr(binding, "paged4_decode", spy_decode)
    assert paged_step.main(["--requests", "3", "--context", "700", "--steps", "2", "--pages", "4", "--bits", "4",
                            "--drafts", str(drafts)]) == 0
    ours = {id(t) for t, _ in turned}
    assert written and asked
    assert all(id(k) in ours for k in written), "keys"
    assert all(id(q) in ours for q in asked), "queries"
    sizes = written[0].float().pow(2).mean(-1)
    assert bool(((sizes - 1).abs() < 0.02).all())  # a norm of 1, in bf16


def test_the_share_is_of_rows_that_see_a_token(cuda, capsys):
    """Requests shorter than a step's verify rows, the first of which see nothing."""
    from sparse_mla_decode_gb300 import paged_step
    assert paged_step.main(["--requests", "40", "--context", "1", "--steps", "1", "--pages", "4", "--bits", "4",
                            "--drafts", "7"]) == 0
    out = capsys.readouterr().out
    assert "100.0% of the attention weight" in out and "nan" not in out
