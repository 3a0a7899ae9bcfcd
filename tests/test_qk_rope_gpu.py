"""smd_qk_norm_rope on the GPU against the 64-bit oracle.

Tolerance. The output is rounded to bf16 once: half a unit, 2^-8 of the value. Before that,
in fp32 (unit 2^-24): the sum of squares of up to 256 columns, at most 16 in a row and 4 joins in a
lane's chain, off by 21 units of itself, half of that in its root; the root's reciprocal (2
units), two products (2): 15 units. A sine or cosine: the angle to 2^-24 of itself, at most pi,
from 32 bits of a turn (2^-31 pi) and of fixed-point frequencies (2^-20 of a turn at the most,
2^-30 for frequencies up to 1), the function's own 2 units: 6 units, plus the turn's.
Products and sum: 3. All in all 24 units of |y_u| + |y_v|: 2^-19, and the turn's error times that."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import paged as opaged
from oracle import paged4 as opaged4
from paged_common import bf16, i32

pytestmark = pytest.mark.gpu


def case(seed, T, H, D, size=1.0):
    rng = np.random.default_rng(seed)
    return opaged.bf16_round(rng.standard_normal((T, H, D)) * size)


def check(got, x, weight, eps, positions, freqs, inter, what=""):
    want, reach = opaged4.qk_norm_rope(x, weight, eps, positions, freqs, inter)
    fast = freqs is not None and np.abs(freqs).max() > 1
    turn = 2 * np.pi * 2.0 ** (-20 if fast else -30)
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -19 + turn) * reach + 1e-38
    err = np.abs(got.float().cpu().numpy().astype(np.float64) - want)
    assert (err <= tol).all(), f"{what}: {(err / tol).max()} of the tolerance"


def frequencies(rng, axes, half, fast=1.0):
    f = np.exp2(-np.arange(half) * 13.0 / half) * fast
    own = rng.integers(0, axes, half)
    return np.where(own == np.arange(axes)[:, None], f, 0.0).astype(np.float32)


@pytest.mark.parametrize("T,Hq,Hk,D,rot,axes,inter,norm", [
    (1, 1, 1, 128, 128, 1, False, True), (1, 64, 8, 128, 128, 1, True, True), (7, 5, 2, 64, 64, 3, False, True),
    (3, 33, 1, 256, 256, 2, False, True), (5, 4, 4, 256, 48, 4, True, True), (13, 3, 1, 128, 64, 1, False, False),
    (2, 40, 40, 64, 16, 2, True, False), (9, 7, 0, 128, 112, 1, False, True), (4, 2, 2, 64, 48, 1, False, True),
    (1500, 3, 1, 128, 128, 3, False, True), (2600, 2, 1, 64, 32, 2, True, True), (701, 9, 2, 256, 256, 1, True, True),
    (700, 2, 1, 256, 16, 4, False, False), (2433, 1, 1, 64, 64, 1, False, True)])
def test_sizes_pairs_and_axes(cuda, T, Hq, Hk, D, rot, axes, inter, norm):
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(T + D + rot)
    q, k = case(1, T, Hq, D, 3.0), case(2, T, Hk, D, 0.2)
    w = [opaged.bf16_round(rng.uniform(0.5, 1.5, D)) if norm else None for _ in "qk"]
    pos = rng.integers(0, [10, 5000, 2 ** 20, 2 ** 31 - 1][axes - 1], (axes, T)).astype(np.int64)
    pos[:, 0] = 0
    f = frequencies(rng, axes, rot // 2)
    one = axes == 1
    got = binding.qk_norm_rope(bf16(q, cuda), bf16(k, cuda) if Hk else None, i32(pos[0] if one else pos, cuda),
                               _f32(f[0] if one else f, cuda), *(None if x is None else bf16(x, cuda) for x in w),
                               eps=1e-5, interleaved=inter)
    check(got[0], q, w[0], 1e-5, pos, f, inter, "q")
    if Hk:
        check(got[1], k, w[1], 1e-5, pos, f, inter, "k")
    else:
        assert got[1] is None


def _f32(x, dev):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(dev)


def test_far_positions_and_fast_and_negative_frequencies(cuda):
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(3)
    T, D = 40, 64
    q = case(4, T, 2, D)
    pos = np.concatenate([2 ** 31 - 1 - np.arange(10), 2 ** np.arange(30)])[None].repeat(2, 0)
    pos[1] = -pos[1]
    for fast in (1.0, 1000.0):
        f = (np.exp2(rng.uniform(-40, 0, (2, 32))) * fast * rng.choice([-1, 1], (2, 32))).astype(np.float32)
        f[0, :4] = [fast, -fast, 1e-40, 0.0]
        got, _ = binding.qk_norm_rope(bf16(q, cuda), None, i32(pos, cuda), _f32(f, cuda))
        check(got, q, None, 0.0, pos, np.where(np.abs(f) < 2.0 ** -126, 0, f).astype(np.float32), False, str(fast))


def test_frequencies_out_of_range_turn_by_nothing(cuda):
    from sparse_mla_decode_gb300 import binding
    q = case(5, 3, 1, 64)
    f = np.zeros((1, 8), dtype=np.float32)
    want = f.copy()
    f[0] = [np.nan, np.inf, -np.inf, 1025.0, 1024.0, -1024.0, 3e38, 0.5]
    want[0, 4:6], want[0, 7] = [1024.0, -1024.0], 0.5
    pos = np.array([[1, 77, 2 ** 31 - 1]])
    got, _ = binding.qk_norm_rope(bf16(q, cuda), None, i32(pos, cuda), _f32(f, cuda))
    check(got, q, None, 0.0, pos, want, False)


@pytest.mark.parametrize("T", [9, 2600])
def test_tokens_with_negative_positions_are_left_alone_also_in_place(cuda, T):
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(T)
    q, k = case(6, T, 3, 64), case(7, T, 1, 64)
    pos = rng.integers(0, 1000, (1, T))
    out = rng.random(T) < 0.4
    out[-1] = True
    pos[0, out] = -1
    f = frequencies(rng, 1, 32)
    w = opaged.bf16_round(rng.uniform(0.5, 1.5, 64))
    # slices of a fused projection, in place, at odd strides
    fused = torch.full((T, 8 * 64), 5.0, dtype=torch.bfloat16, device=cuda)
    fused[:, 64:256], fused[:, 320:384] = bf16(q, cuda).flatten(1), bf16(k, cuda).flatten(1)
    tq, tk = fused[:, 64:256].view(T, 3, 64), fused[:, 320:384].view(T, 1, 64)
    got = binding.qk_norm_rope(tq, tk, i32(pos[0], cuda), _f32(f[0], cuda), bf16(w, cuda), bf16(w, cuda),
                               q_out=tq, k_out=tk)
    assert got[0].data_ptr() == tq.data_ptr()
    for t, x in ((tq, q), (tk, k)):
        assert np.array_equal(t[out.tolist()].float().cpu().numpy(), x[out])
        live = ~out
        check(t[live.tolist()], x[live], w, 1e-6, pos[:, live], f, False)
    for a, b in ((0, 64), (256, 320), (384, 512)):
        assert bool((fused[:, a:b] == 5.0).all())


def test_norm_of_zeros_extremes_nans_and_without_rotation(cuda):
    import torch
    from sparse_mla_decode_gb300 import binding
    x = case(8, 8, 2, 128)
    x[0], x[1] = 0.0, opaged.bf16_round(x[1] * 2.0 ** 50)
    x[2] = opaged.bf16_round(x[2] * 2.0 ** -50)
    x[3, 0] = 2.0 ** -130
    w = opaged.bf16_round(np.linspace(-2, 2, 128))
    got, _ = binding.qk_norm_rope(bf16(x, cuda), None, None, None, bf16(w, cuda), eps=1e-6)
    check(got, x, w, float(np.float32(1e-6)), None, None, False)
    y = x.copy()
    y[5, 1, 3], y[6, 0, 9] = np.nan, np.inf
    got, _ = binding.qk_norm_rope(bf16(y, cuda), None, None, None, bf16(w, cuda))
    nan = torch.isnan(got).any(-1).cpu().numpy()
    assert nan[5].tolist() == [False, True] and nan[6].tolist() == [True, False] and nan.sum() == 2
    same, _ = binding.qk_norm_rope(bf16(x, cuda), None, None, None)
    assert torch.equal(same, bf16(x, cuda))
    none = binding.qk_norm_rope(torch.empty((0, 2, 64), dtype=torch.bfloat16, device=cuda), None,
                                torch.empty(0, dtype=torch.int32, device=cuda), torch.ones(32, device=cuda))
    assert none[0].shape == (0, 2, 64)


def test_many_heads_another_stream_and_a_graph(cuda):
    import torch
    from sparse_mla_decode_gb300 import binding
    rng = np.random.default_rng(9)
    q, k = case(10, 3, 300, 128), case(11, 3, 77, 128)
    pos = np.array([[3, 100000, 7], [5, 6, 7]])
    f = frequencies(rng, 2, 64)
    args = bf16(q, cuda), bf16(k, cuda), i32(pos, cuda), _f32(f, cuda)
    out = binding.qk_norm_rope(*args)
    check(out[0], q, None, 0, pos, f, False)
    check(out[1], k, None, 0, pos, f, False)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = binding.qk_norm_rope(*args, stream=side)
    side.synchronize()
    assert torch.equal(out[0], other[0]) and torch.equal(out[1], other[1])
    buf = [torch.zeros_like(t) for t in out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.qk_norm_rope(*args, q_out=buf[0], k_out=buf[1])
    pos[0] = [9, 1, 2]
    args[2].copy_(i32(pos, cuda))
    graph.replay()
    torch.cuda.synchronize()
    check(buf[0], q, None, 0, pos, f, False)
    check(buf[1], k, None, 0, pos, f, False)


@pytest.mark.parametrize("T,Hq,Hk,D,rot,axes,inter,norm", [
    (5000, 3, 1, 128, 32, 2, False, True), (9800, 2, 1, 64, 16, 1, True, False), (2501, 2, 1, 256, 16, 3, False, True),
    (4900, 19, 0, 128, 16, 1, True, True), (4900, 18, 2, 128, 16, 1, False, True)])
def test_many_tokens_of_few_heads(cuda, T, Hq, Hk, D, rot, axes, inter, norm):
    test_sizes_pairs_and_axes(cuda, T, Hq, Hk, D, rot, axes, inter, norm)


def test_negative_positions_among_many_tokens_of_few_heads(cuda):
    test_tokens_with_negative_positions_are_left_alone_also_in_place(cuda, 9800)
