"""smd_verify_drafts on the GPU against whole numbers and fractions: every output is equal."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import paged4 as opaged4
from paged_common import i32

pytestmark = pytest.mark.gpu


def f32(x, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(dev)


def distributions(rng, R, G, V, sharp=2.0, apart=0.5):
    x = rng.standard_normal((R, G, V)) * sharp
    y = x[:, :G - 1] + apart * rng.standard_normal((R, G - 1, V))

    def softmax(z):
        e = np.exp(z - z.max(-1, keepdims=True)) if z.size else z
        return (e / e.sum(-1, keepdims=True)).astype(np.float32) if z.size else z.astype(np.float32)
    return softmax(x), softmax(y)


def drawn(rng, q):
    R, n, V = q.shape
    c = q.cumsum(-1)
    u = rng.random((R, n, 1)) * c[..., -1:] if n else np.zeros((R, 0, 1))
    return (c < u).sum(-1).clip(0, V - 1)


def check(cuda, p, q, tokens, accept, sample, **kw):
    import torch
    from sparse_mla_decode_gb300 import binding
    gp = p if isinstance(p, torch.Tensor) else f32(p, cuda)
    gq = q if q is None or isinstance(q, torch.Tensor) else f32(q, cuda)
    got = binding.verify_drafts(gp, i32(tokens, cuda), f32(accept, cuda), f32(sample, cuda), draft=gq, **kw)
    torch.cuda.synchronize()
    p, q = (x.cpu().numpy() if isinstance(x, torch.Tensor) else x for x in (p, q))
    want = opaged4.verify_drafts(p, q, tokens, accept.astype(np.float32), sample.astype(np.float32))
    for name, a, b in zip(("tokens", "accepted", "rejected"), got, want):
        assert np.array_equal(a.cpu().numpy().astype(np.int64), b), name
    return want


@pytest.mark.parametrize("R,G,V", [(1, 4, 1), (3, 2, 2), (40, 3, 33), (7, 4, 1003), (64, 8, 129), (5, 1, 5000),
                                   (2, 64, 257), (3, 5, 32768), (2, 3, 100003), (300, 4, 640), (1, 2, 262144)])
@pytest.mark.parametrize("given", [True, False])
def test_batches(cuda, R, G, V, given):
    rng = np.random.default_rng(R + G + V)
    p, q = distributions(rng, R, G, V)
    tokens = drawn(rng, q)
    accept, sample = rng.random((R, G - 1)), rng.random(R)
    if not given and V > 100:  # likely tokens, or none would stay
        tokens = p[:, :G - 1].argmax(-1)
        accept = accept * 0.05
    check(cuda, p, q if given and G > 1 else None, tokens, accept, sample)


def test_every_place_that_a_draw_can_fall_on(cuda):
    """Probabilities in whole multiples of 2^-12 over rows cut at warps, CTAs and lanes: each border
    of the sums, just below and on it."""
    rng = np.random.default_rng(1)
    for V in (5, 700, 9000):
        at = np.unique(np.concatenate([rng.integers(0, V, 30), [0, V - 1], np.arange(0, V, 128)[:40], np.arange(0, V, 1024)]))
        share = rng.multinomial(4096 - len(at), np.ones(len(at)) / len(at)) + 1
        p = np.zeros(V, dtype=np.float32)
        p[at] = share / 4096
        c = np.cumsum(share) / 4096
        u = np.concatenate([[0.0], c[:-1], c - 2.0 ** -24, [np.nextafter(np.float32(1), np.float32(0))]])
        R = len(u)
        want = check(cuda, np.tile(p, (R, 1, 1)), None, np.zeros((R, 0), dtype=int), np.zeros((R, 0)), u)
        assert set(want[0][:, 0]) == set(at)


def test_the_residual_is_of_the_first_refused_token(cuda):
    """Refusals at every place, and none; a border of the test itself (u q = p is refused)."""
    rng = np.random.default_rng(2)
    G, V = 6, 300
    R = 2 * G
    p, q = distributions(rng, R, G, V)
    tokens = drawn(rng, q)
    accept = np.zeros((R, G - 1))
    row = np.arange(R)
    for r in row[:G - 1]:
        d = tokens[r, r]
        p[r, r, d], q[r, r, d], accept[r, r] = 0.25, 0.5, 0.5
    for r in row[G:R - 1]:
        d = tokens[r, r - G]
        p[r, r - G, d], q[r, r - G, d], accept[r, r - G] = 0.25, 0.5, np.nextafter(np.float32(0.5), np.float32(0))
    want = check(cuda, p, q, tokens, accept, rng.random(R))
    assert want[1].tolist() == [0, 1, 2, 3, 4, 5] + [5] * 6


def test_drafts_that_end_early_and_tokens_outside(cuda):
    rng = np.random.default_rng(3)
    R, G, V = 9, 5, 2000
    p, q = distributions(rng, R, G, V)
    tokens = drawn(rng, q)
    for r, bad in enumerate([-1, V, 2 ** 31 - 1, -2 ** 31, -5]):
        tokens[r, r % 4:] = bad
    accept = np.zeros((R, G - 1))
    for given in (q, None):
        want = check(cuda, p, given, tokens, accept, rng.random(R))
        assert want[1][:5].tolist() == [0, 1, 2, 3, 0]


def test_rows_without_anything_to_draw(cuda):
    """A residual of zeros falls back to the target; a target of zeros gives -1."""
    rng = np.random.default_rng(4)
    R, G, V = 8, 3, 5000
    p, q = distributions(rng, R, G, V)
    tokens, accept, sample = drawn(rng, q), np.ones((R, G - 1)), rng.random(R)
    p[0, 0] = q[0, 0]                       # nothing left
    p[1, 0], q[1, 0] = 0.0, q[1, 0]
    p[2], q[2] = 0.0, 0.0
    p[3, 0], q[3, 0] = 2.0 ** -41, 0.0     # below the unit, and stays
    p[4, 0], q[4, 0] = 0.0, 0.0
    p[4, 0, 4999] = 2.0 ** -40
    p[5, 0], q[5, 0] = 0.0, 1.0
    p[5, 0, tokens[5, 0]] = 0.5
    want = check(cuda, p, q, tokens, accept, sample)
    assert want[0][1, 0] == -1 and want[0][2, 0] == -1 and want[1][3] >= 1
    assert want[0][5, 0] == tokens[5, 0]
    p[7, 0] = q[7, 0] = 2.0 ** -41
    want = check(cuda, p, q, tokens, accept, sample)
    assert want[0][7, 0] == -1
    p[6, 0] = 0.0
    p[6, 0, tokens[6, 0]] = 1.0
    check(cuda, p, None, tokens, accept, sample)


def test_nans_infinities_and_random_numbers_out_of_range(cuda):
    rng = np.random.default_rng(5)
    R, G, V = 12, 4, 3000
    p, q = distributions(rng, R, G, V)
    tokens = drawn(rng, q)
    accept, sample = rng.random((R, G - 1)), rng.random(R)
    p[0, 0, ::7], q[0, 0, 5], p[1, 0, 3], q[1, 1, 9] = np.nan, np.nan, np.inf, np.inf
    p[2, 0], p[2, 0, 17] = -1.0, 7.0
    p[3, 0, tokens[3, 0]], q[4, 0, tokens[4, 0]] = np.nan, np.nan
    accept[5, 0], accept[6, 0], accept[7, 0], accept[8, 0] = np.nan, np.inf, -1.0, 2.0
    sample[5:12] = [np.nan, np.inf, -np.inf, 1.0, 2.0, -0.5, 1e-30]
    check(cuda, p, q, tokens, accept, sample)
    check(cuda, p, None, tokens, accept, sample)


@pytest.mark.parametrize("V,pad,off", [(1001, 0, 0), (1000, 0, 0), (1000, 3, 0), (1000, 8, 1), (4096, 4, 4)])
def test_strides_and_alignments(cuda, V, pad, off):
    import torch
    rng = np.random.default_rng(V + pad)
    R, G = 5, 3
    p, q = distributions(rng, R, G, V)
    tokens, accept, sample = drawn(rng, q), rng.random((R, G - 1)), rng.random(R)

    def apart(x):
        n = x.shape[0] * x.shape[1]
        flat = torch.full((n * (V + pad) + off,), float("nan"), device=cuda)
        v = flat[off:].view(n, V + pad)[:, :V].view(x.shape[0], x.shape[1], V) if pad == 0 else \
            flat[off:].as_strided(x.shape, (x.shape[1] * (V + pad), V + pad, 1), off)
        v.copy_(f32(x, cuda))
        return v
    check(cuda, apart(p), apart(q), tokens, accept, sample)


def test_more_requests_than_a_grid_row_and_a_graph(cuda):
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(6)
    R, G, V = 65535 + 70, 2, 5
    p, q = distributions(rng, 50, G, V)
    p, q = np.tile(p, (R // 50 + 1, 1, 1))[:R], np.tile(q, (R // 50 + 1, 1, 1))[:R]
    tokens, accept, sample = drawn(rng, q), rng.random((R, 1)), rng.random(R)
    got = binding.verify_drafts(f32(p, cuda), i32(tokens, cuda), f32(accept, cuda), f32(sample, cuda), draft=f32(q, cuda))
    pick = np.r_[0:40, 65500:65570, R - 20:R]
    want = opaged4.verify_drafts(p[pick], q[pick], tokens[pick], accept[pick].astype(np.float32), sample[pick].astype(np.float32))
    for a, b in zip(got, want):
        assert np.array_equal(a.cpu().numpy()[pick], b)
    args = [f32(p[:64], cuda), i32(tokens[:64], cuda), f32(accept[:64], cuda), f32(sample[:64], cuda)]
    out = dict(out_tokens=torch.zeros((64, 2), dtype=torch.int32, device=cuda),
               accepted=torch.zeros(64, dtype=torch.int32, device=cuda),
               rejected=torch.zeros(64, dtype=torch.int32, device=cuda))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        binding.verify_drafts(*args, draft=f32(q[:64], cuda), **out)
    side.synchronize()
    assert torch.equal(out["out_tokens"], got[0][:64])
    dq = f32(q[:64], cuda)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.verify_drafts(*args, draft=dq, **out)
    args[3].copy_(f32(sample[64:128], cuda))
    graph.replay()
    torch.cuda.synchronize()
    want = opaged4.verify_drafts(p[:64], q[:64], tokens[:64], accept[:64].astype(np.float32), sample[64:128].astype(np.float32))
    assert np.array_equal(out["out_tokens"].cpu().numpy(), want[0])


def test_sampling_follows_the_target(cuda):
    """Drafts from q, then the call: the first tokens' frequencies are the target's, within 5 standard
    deviations of each count."""
    import torch
    from sparse_mla_decode_gb300 import binding
    R, V = 200000, 16
    g = torch.Generator(device=cuda).manual_seed(7)
    p, q = (torch.softmax(torch.randn(V, generator=g, device=cuda) * 1.5, -1) for _ in "pq")
    d = torch.multinomial(q, R, replacement=True, generator=g).int()[:, None]
    u = torch.rand(R, 1, generator=g, device=cuda)
    s = torch.rand(R, generator=g, device=cuda)
    out, _, _ = binding.verify_drafts(p.expand(R, 2, V).contiguous(), d, u, s, draft=q.expand(R, 1, V).contiguous())
    n = torch.bincount(out[:, 0].long(), minlength=V).double()
    dev = (R * p.double() * (1 - p.double())).sqrt()
    assert bool(((n - R * p.double()).abs() <= 5 * dev + 1).all())
