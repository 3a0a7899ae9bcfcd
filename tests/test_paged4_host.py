"""The 4-bit cache and the step around it without a GPU: the oracle against closed forms,
and the refusals that come before any launch."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest

from oracle import paged as opaged
from oracle import paged4 as opaged4
from sparse_mla_decode_gb300 import binding as smd
from test_paged_host import OnGpu, two_gpus  # noqa: F401  (a fixture)

A = 1 << 20  # an aligned address that nothing is read from


# ---- the oracle ------------------------------------------------------------------------------

def test_e2m1_codes():
    """Sign, two exponent bits (bias 1), one mantissa bit."""
    for c in range(16):
        e, m = c >> 1 & 3, c & 1
        v = (m / 2 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)) * (-1 if c & 8 else 1)
        assert opaged4.VALUES[c] == v
    got = opaged4.e2m1_encode(np.array([0.25, 0.26, 0.75, 0.74, 1.25, 1.75, 2.5, 2.51, 3.5, 5.0, 5.01, 1e9, -0.3, -0.2]))
    assert got.tolist() == [0, 1, 2, 1, 2, 4, 4, 5, 6, 6, 7, 7, 9, 0]
    c = np.arange(32, dtype=np.uint8).reshape(2, 16) % 16
    assert np.array_equal(opaged4.unpack(opaged4.pack(c)), c) and opaged4.pack(c)[0, 0] == 0x10


def test_quantised_values_are_near_and_blocks_are_apart():
    rng = np.random.default_rng(0)
    x = opaged.bf16_round(rng.standard_normal((50, 2, 64)) * np.exp2(rng.integers(-2, 6, (50, 2, 1))))
    c, s = opaged4.quantise(x, [3, -2])
    v = opaged4.VALUES[opaged4.unpack(c)].reshape(50, 2, 4, 16) * opaged.VALUES[s][..., None]
    v = v.reshape(x.shape) * np.exp2([3.0, -2.0])[:, None]
    a = np.abs(x).reshape(50, 2, 4, 16).max(-1).repeat(16, -1)
    # a step between 4 and 6 of a scale that is off by 2^-4 at most, or the largest cut at 6 of it
    assert (np.abs(v - x) <= a * (1 / 6 * (1 + 2.0 ** -4) + 2.0 ** -4)).all()
    y = x.copy()
    y[7, 1, 16:32] *= 4
    c2, s2 = opaged4.quantise(y, [3, -2])
    same = np.ones(c.shape, dtype=bool)
    same[7, 1, 8:16] = False
    assert np.array_equal(c[same], c2[same]) and (s2 != s).sum() == 1


def test_read_of_quantised_values_is_bf16_exact():
    v = opaged4.GRID[:, None] * opaged.VALUES[None, :127]
    assert np.array_equal(opaged.bf16_round(v), v)
    assert np.array_equal(v.astype(np.float16).astype(np.float64), v)


def test_attention_oracle_of_equal_logits_is_the_mean():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((2, 3, 1, 16, 64))
    table = np.array([[2, 0], [1, 1]])
    out, lse, _, _ = opaged4.attend(np.zeros((2, 1, 64)), k, v, table, [20, 0], 0.1)
    assert np.allclose(out[0, 0], np.concatenate([v[2, 0], v[0, 0, :4]]).mean(0)) and np.isclose(lse[0, 0], np.log(20))
    assert (out[1] == 0).all() and np.isneginf(lse[1]).all()


def test_rotation_oracle():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((4, 2, 64))
    f = np.array([[0.5] * 8, [0.0] * 7 + [0.25]])
    pos = np.array([[0, 1, 2, 2 ** 30], [4, 4, 0, -3]])
    for inter in (False, True):
        y, _ = opaged4.qk_norm_rope(x, None, 0.0, pos, f, inter)
        u, v = (2 * 7, 2 * 7 + 1) if inter else (7, 15)
        z = (x[2, 1, u] + 1j * x[2, 1, v]) * np.exp(1j * (2 * 0.5))
        assert np.allclose([y[2, 1, u], y[2, 1, v]], [z.real, z.imag])
        assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
        assert np.array_equal(y[..., 16:], x[..., 16:])
        assert np.allclose(y[0, 0, [0, 2]], x[0, 0, [0, 2]])  # position 0, pairs that axis 1 leaves alone
        z = (x[3, 0, u] + 1j * x[3, 0, v]) * np.exp(1j * math.remainder(2 ** 29 - 0.75, 2 * math.pi))
        assert np.allclose([y[3, 0, u], y[3, 0, v]], [z.real, z.imag], atol=1e-6)
    y, _ = opaged4.qk_norm_rope(x, np.full(64, 2.0), 0.0, None, None, False)
    assert np.allclose((y * y).mean(-1), 4.0)


def test_verify_oracle_keeps_the_targets_distribution():
    """Over all first tokens and a grid of both random numbers, token v comes out p(v) of the time."""
    p, q = np.float32([0.5, 0.25, 0.125, 0.125]), np.float32([0.125, 0.5, 0.25, 0.125])
    n, freq = 32, np.zeros(4)
    grid = (np.arange(n) + 0.5) / n
    for d in range(4):
        u, s = (x.ravel().astype(np.float32) for x in np.meshgrid(grid, grid))
        R = len(u)
        out, a, rej = opaged4.verify_drafts(np.tile(p, (R, 2, 1)), np.tile(q, (R, 1, 1)), np.full((R, 1), d), u[:, None], s)
        assert np.array_equal(a + rej, np.ones(R)) and ((out[:, 1] >= 0) == (a == 1)).all()
        freq += q[d] * np.bincount(out[:, 0], minlength=4) / R
    assert np.abs(freq - p).max() <= 1 / n
    out, a, _ = opaged4.verify_drafts(np.tile(p, (3, 3, 1)), None, np.array([[0, -1], [9, 0], [0, 1]]),
                                      np.zeros((3, 2)), np.zeros(3))
    assert a.tolist() == [1, 0, 2] and out.tolist() == [[0, 0, -1], [0, -1, -1], [0, 1, 0]]


def test_trim_oracle():
    table = np.arange(12).reshape(3, 4) + 100
    new, state, ring = opaged4.block_trim([60, 17, 5], [30, 1, 0], table, np.zeros(10, dtype=int), [3, 9], 16)
    assert new.tolist() == [30, 16, 5] and state.tolist() == [3, 12]
    assert ring.tolist() == [103, 105, 0, 0, 0, 0, 0, 0, 0, 102]


# ---- refusals --------------------------------------------------------------------------------

KV4 = dict(k=A, v=A, k_scales=A, v_scales=A, k_stride=(4096, 2048, 64), v_stride=(4096, 2048, 64), bounds=A,
           pages=10, heads=2, page_size=32, head_dim=128)


def cache(**kw):
    c = smd.SmdPagedCache4()
    for name, v in {**KV4, **kw}.items():
        setattr(c, name, (ctypes.c_int64 * 3)(*v) if name.endswith("stride") else v)
    return c


@pytest.mark.parametrize("kw,code", [
    (dict(k=0), smd.SMD_ERR_NULL), (dict(v=0), smd.SMD_ERR_NULL), (dict(k_scales=0), smd.SMD_ERR_NULL),
    (dict(v_scales=0), smd.SMD_ERR_NULL), (dict(pages=0), smd.SMD_ERR_SHAPE), (dict(heads=0), smd.SMD_ERR_SHAPE),
    (dict(heads=65536), smd.SMD_ERR_SHAPE), (dict(page_size=8), smd.SMD_ERR_SHAPE),
    (dict(page_size=40), smd.SMD_ERR_SHAPE), (dict(page_size=272), smd.SMD_ERR_SHAPE),
    (dict(head_dim=96), smd.SMD_ERR_SHAPE), (dict(pages=2 ** 26), smd.SMD_ERR_SHAPE),
    (dict(k_stride=(4096, 2048, 48)), smd.SMD_ERR_SHAPE), (dict(v_stride=(4096, -2048, 64)), smd.SMD_ERR_SHAPE),
    (dict(v_stride=(2 ** 40, 2048, 64)), smd.SMD_ERR_SHAPE), (dict(k_stride=(4096, 2048, 72)), smd.SMD_ERR_ALIGN),
    (dict(k=A + 8), smd.SMD_ERR_ALIGN), (dict(v=A + 4), smd.SMD_ERR_ALIGN), (dict(k_scales=A + 8), smd.SMD_ERR_ALIGN),
    (dict(v_scales=A + 1), smd.SMD_ERR_ALIGN), (dict(k_exp=A + 2), smd.SMD_ERR_ALIGN),
    (dict(v_exp=A + 1), smd.SMD_ERR_ALIGN), (dict(bounds=A + 8), smd.SMD_ERR_ALIGN)])
def test_cache_description(kw, code):
    assert smd.lib().smd_paged4_cache_init(ctypes.byref(cache(**kw))) == code


def test_a_null_or_unfinished_cache_is_refused():
    so, c = smd.lib(), cache()
    ref = ctypes.byref(c)
    assert so.smd_paged4_cache_init(None) == smd.SMD_ERR_NULL
    assert so.smd_paged4_workspace_bytes(None) == smd.SMD_ERR_NULL
    assert so.smd_paged4_workspace_bytes(ref) == smd.SMD_ERR_PLAN
    assert so.smd_paged4_append(None, A, 256, A, 256, A, 1, 0) == smd.SMD_ERR_NULL
    assert so.smd_paged4_append(ref, A, 256, A, 256, A, 1, 0) == smd.SMD_ERR_PLAN
    assert so.smd_paged4_read(None, A, 1, A, 256, A, 256, 0) == smd.SMD_ERR_NULL
    assert so.smd_paged4_read(ref, A, 1, A, 256, A, 256, 0) == smd.SMD_ERR_PLAN
    rows = (A, 512, ref, A, 4, 4, A, 2, 1, 4)
    assert so.smd_paged4_decode(*rows, 0.1, None, None, 0, A, A, None, A, 1 << 30, 0) == smd.SMD_ERR_PLAN
    assert so.smd_paged4_decode(A, 512, None, *rows[3:], 0.1, None, None, 0, A, A, None, A, 1 << 30, 0) == smd.SMD_ERR_NULL


def finished():
    """A description that says it is finished: the refusals after that need no descriptors."""
    c = cache()
    c.map[0] = 0x736d645061673465
    return c


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), smd.SMD_OK), (dict(T=-1), smd.SMD_ERR_SHAPE), (dict(k_stride=255), smd.SMD_ERR_SHAPE),
    (dict(v_stride=260), smd.SMD_ERR_SHAPE), (dict(k=0), smd.SMD_ERR_NULL), (dict(v=0), smd.SMD_ERR_NULL),
    (dict(slots=0), smd.SMD_ERR_NULL), (dict(k=A + 8), smd.SMD_ERR_ALIGN), (dict(v=A + 2), smd.SMD_ERR_ALIGN),
    (dict(slots=A + 2), smd.SMD_ERR_ALIGN)])
def test_append(kw, code):
    f = {**dict(k=A, k_stride=256, v=A, v_stride=256, slots=A, T=3), **kw}
    assert smd.lib().smd_paged4_append(ctypes.byref(finished()), *f.values(), 0) == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), smd.SMD_OK), (dict(k=0, v=0), smd.SMD_OK), (dict(T=-1), smd.SMD_ERR_SHAPE),
    (dict(k_stride=255), smd.SMD_ERR_SHAPE), (dict(v_stride=260), smd.SMD_ERR_SHAPE), (dict(slots=0), smd.SMD_ERR_NULL),
    (dict(k=A + 8), smd.SMD_ERR_ALIGN), (dict(v=A + 2), smd.SMD_ERR_ALIGN), (dict(slots=A + 2), smd.SMD_ERR_ALIGN)])
def test_read(kw, code):
    f = {**dict(slots=A, T=3, k=A, k_stride=256, v=A, v_stride=256), **kw}
    assert smd.lib().smd_paged4_read(ctypes.byref(finished()), *f.values(), 0) == code


@pytest.mark.parametrize("kw,code", [
    (dict(R=0), smd.SMD_OK), (dict(R=-1), smd.SMD_ERR_SHAPE), (dict(G=0), smd.SMD_ERR_SHAPE), (dict(G=9), smd.SMD_ERR_SHAPE),
    (dict(Hq=3), smd.SMD_ERR_SHAPE), (dict(Hq=258), smd.SMD_ERR_SHAPE), (dict(width=0), smd.SMD_ERR_SHAPE),
    (dict(table_stride=3), smd.SMD_ERR_SHAPE), (dict(q_stride=516), smd.SMD_ERR_SHAPE), (dict(q=0), smd.SMD_ERR_NULL),
    (dict(lists=A, K=-1), smd.SMD_ERR_SHAPE), (dict(lists=A, K=2 ** 26), smd.SMD_ERR_SHAPE),
    (dict(out=0), smd.SMD_ERR_NULL), (dict(ws=0), smd.SMD_ERR_NULL), (dict(out=A + 8), smd.SMD_ERR_ALIGN),
    (dict(lse=A + 2), smd.SMD_ERR_ALIGN), (dict(q=A + 8), smd.SMD_ERR_ALIGN)])
def test_decode(kw, code):
    f = {**dict(q=A, q_stride=512, c=ctypes.byref(finished()), table=A, table_stride=4, width=4, lengths=A, R=2, G=1, Hq=4,
                sm=0.1, lists=0, counts=0, K=0, out=A, lse=A, status=0, ws=A, bytes=1 << 30), **kw}
    assert smd.lib().smd_paged4_decode(*f.values(), 0) == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), smd.SMD_OK), (dict(T=-1), smd.SMD_ERR_SHAPE), (dict(T=2 ** 30, pos_stride=2 ** 30), smd.SMD_ERR_SHAPE),
    (dict(D=96), smd.SMD_ERR_SHAPE), (dict(Hq=0), smd.SMD_ERR_SHAPE), (dict(Hk=-1), smd.SMD_ERR_SHAPE),
    (dict(rot=24), smd.SMD_ERR_SHAPE), (dict(rot=144), smd.SMD_ERR_SHAPE), (dict(rot=-16), smd.SMD_ERR_SHAPE),
    (dict(axes=0), smd.SMD_ERR_SHAPE), (dict(axes=5), smd.SMD_ERR_SHAPE), (dict(eps=-1.0), smd.SMD_ERR_SHAPE),
    (dict(eps=math.nan), smd.SMD_ERR_SHAPE), (dict(eps=math.inf), smd.SMD_ERR_SHAPE), (dict(q_stride=511), smd.SMD_ERR_SHAPE),
    (dict(q_stride=516), smd.SMD_ERR_SHAPE), (dict(k_stride=252), smd.SMD_ERR_SHAPE), (dict(qo_stride=504), smd.SMD_ERR_SHAPE),
    (dict(ko_stride=260), smd.SMD_ERR_SHAPE), (dict(pos_stride=4), smd.SMD_ERR_SHAPE), (dict(q=0), smd.SMD_ERR_NULL),
    (dict(k=0), smd.SMD_ERR_NULL), (dict(qo=0), smd.SMD_ERR_NULL), (dict(ko=0), smd.SMD_ERR_NULL),
    (dict(pos=0), smd.SMD_ERR_NULL), (dict(freqs=0), smd.SMD_ERR_NULL), (dict(q=A + 8), smd.SMD_ERR_ALIGN),
    (dict(k=A + 2), smd.SMD_ERR_ALIGN), (dict(qw=A + 8), smd.SMD_ERR_ALIGN), (dict(kw=A + 4), smd.SMD_ERR_ALIGN),
    (dict(qo=A + 8), smd.SMD_ERR_ALIGN), (dict(ko=A + 8), smd.SMD_ERR_ALIGN), (dict(pos=A + 2), smd.SMD_ERR_ALIGN),
    (dict(freqs=A + 1), smd.SMD_ERR_ALIGN)])
def test_rope(kw, code):
    f = {**dict(q=A, q_stride=512, k=A, k_stride=256, T=5, Hq=4, Hk=2, D=128, pos=A, pos_stride=5, axes=1, freqs=A,
                rot=128, inter=0, qw=A, kw=A, eps=1e-6, qo=A, qo_stride=512, ko=A, ko_stride=256), **kw}
    assert smd.lib().smd_qk_norm_rope(*f.values(), 0) == code


@pytest.mark.parametrize("kw,code", [
    (dict(R=0), smd.SMD_OK), (dict(R=-1), smd.SMD_ERR_SHAPE), (dict(G=0), smd.SMD_ERR_SHAPE), (dict(G=65), smd.SMD_ERR_SHAPE),
    (dict(V=0), smd.SMD_ERR_SHAPE), (dict(V=2 ** 22 + 1, ts=2 ** 23, ds=2 ** 23), smd.SMD_ERR_SHAPE),
    (dict(ts=99), smd.SMD_ERR_SHAPE), (dict(ds=99), smd.SMD_ERR_SHAPE), (dict(R=2 ** 29, G=4), smd.SMD_ERR_SHAPE),
    (dict(target=0), smd.SMD_ERR_NULL), (dict(tokens=0), smd.SMD_ERR_NULL), (dict(accept=0), smd.SMD_ERR_NULL),
    (dict(sample=0), smd.SMD_ERR_NULL), (dict(out=0), smd.SMD_ERR_NULL), (dict(target=A + 2), smd.SMD_ERR_ALIGN),
    (dict(draft=A + 1), smd.SMD_ERR_ALIGN), (dict(tokens=A + 2), smd.SMD_ERR_ALIGN), (dict(accepted=A + 2), smd.SMD_ERR_ALIGN)])
def test_verify(kw, code):
    f = {**dict(target=A, ts=100, draft=A, ds=100, tokens=A, accept=A, sample=A, R=3, G=4, V=100, out=A, accepted=A,
                rejected=A), **kw}
    assert smd.lib().smd_verify_drafts(*f.values(), 0) == code


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), smd.SMD_ERR_SHAPE), (dict(R=8193), smd.SMD_ERR_SHAPE), (dict(pages=0), smd.SMD_ERR_SHAPE),
    (dict(P=0), smd.SMD_ERR_SHAPE), (dict(width=0), smd.SMD_ERR_SHAPE), (dict(stride=3), smd.SMD_ERR_SHAPE),
    (dict(pages=2 ** 30, P=2), smd.SMD_ERR_SHAPE), (dict(width=2 ** 28, stride=2 ** 28), smd.SMD_ERR_SHAPE),
    (dict(lengths=0), smd.SMD_ERR_NULL), (dict(drop=0), smd.SMD_ERR_NULL), (dict(table=0), smd.SMD_ERR_NULL),
    (dict(ring=0), smd.SMD_ERR_NULL), (dict(state=0), smd.SMD_ERR_NULL), (dict(new_lengths=0), smd.SMD_ERR_NULL),
    (dict(new_state=0), smd.SMD_ERR_NULL), (dict(drop=A + 2), smd.SMD_ERR_ALIGN), (dict(state=A + 4), smd.SMD_ERR_ALIGN)])
def test_trim(kw, code):
    f = {**dict(lengths=A, drop=A, R=2, table=A, stride=4, width=4, ring=A, pages=8, state=A, P=16, new_lengths=A,
                new_state=A), **kw}
    assert smd.lib().smd_block_trim(*f.values(), 0) == code


# ---- the binding: which GPU, and what it refuses ---------------------------------------------

def calls():
    """Each call's tensors by name, and the call on them."""
    import torch

    def zeros(*shape, dtype=torch.int32):
        return torch.zeros(shape, dtype=dtype)

    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    pool = dict(k=zeros(4, 2, 16, 32, dtype=u8), v=zeros(4, 2, 16, 32, dtype=u8), k_scales=zeros(4, 2, 16, 4, dtype=u8),
                v_scales=zeros(4, 2, 16, 4, dtype=u8), k_exp=zeros(2), v_exp=zeros(2), bounds=zeros(4, 2, 2, 64, dtype=bf))
    tokens = dict(k_new=zeros(5, 2, 64, dtype=bf), v_new=zeros(5, 2, 64, dtype=bf), slots=zeros(5))

    def on_cache(call):
        def with_cache(**t):
            c = smd.PagedCache4(**{n: t.pop(n) for n in pool})
            call(c, t)
        return with_cache

    return {
        "smd_paged4_append": (dict(pool, **tokens),
                              on_cache(lambda c, t: smd.paged4_append(c, t["k_new"], t["v_new"], t["slots"], stream=7))),
        "smd_paged4_read": (dict(pool, **tokens),
                            on_cache(lambda c, t: smd.paged4_read(c, t["slots"], t["k_new"], t["v_new"], stream=7))),
        "smd_paged4_decode": (dict(pool, q=zeros(3, 4, 64, dtype=bf), table=zeros(3, 2), lengths=zeros(3),
                                   block_lists=zeros(3, 2, 1), block_counts=zeros(3, 2), out=zeros(3, 4, 64, dtype=bf),
                                   lse=zeros(3, 4, dtype=f32), status=zeros(1), workspace=zeros(16, dtype=u8)),
                              on_cache(lambda c, t: smd.paged4_decode(cache=c, sm_scale=0.1, stream=7, **t))),
        "smd_block_scores": (dict(pool, q=zeros(3, 4, 64, dtype=bf), table=zeros(3, 2), lengths=zeros(3),
                                  out=zeros(3, 2, 2, dtype=bf)),
                             on_cache(lambda c, t: smd.block_scores(cache=c, stream=7, **t))),
        "smd_qk_norm_rope": (dict(q=zeros(5, 4, 64, dtype=bf), k=zeros(5, 2, 64, dtype=bf), positions=zeros(3, 5),
                                  freqs=zeros(3, 32, dtype=f32), q_weight=zeros(64, dtype=bf), k_weight=zeros(64, dtype=bf),
                                  q_out=zeros(5, 4, 64, dtype=bf), k_out=zeros(5, 2, 64, dtype=bf)),
                             lambda **t: smd.qk_norm_rope(stream=7, **t)),
        "smd_verify_drafts": (dict(target=zeros(3, 4, 10, dtype=f32), tokens=zeros(3, 3), accept=zeros(3, 3, dtype=f32),
                                   sample=zeros(3, dtype=f32), draft=zeros(3, 3, 10, dtype=f32), out_tokens=zeros(3, 4),
                                   accepted=zeros(3), rejected=zeros(3)),
                              lambda **t: smd.verify_drafts(stream=7, **t)),
        "smd_block_trim": (dict(lengths=zeros(3), drop=zeros(3), table=zeros(3, 2), ring=zeros(4),
                                state=zeros(2, dtype=torch.int64), new_lengths=zeros(3),
                                new_state=zeros(2, dtype=torch.int64)),
                           lambda **t: smd.block_trim(page_size=16, stream=7, **t))}


@pytest.mark.parametrize("name", list(calls()))
@pytest.mark.parametrize("index", [0, 1])
def test_a_call_runs_on_the_gpu_of_its_tensors(two_gpus, name, index):  # noqa: F811
    tensors, call = calls()[name]
    call(**{n: OnGpu(t, index) for n, t in tensors.items()})
    assert (name, index) in two_gpus


@pytest.mark.parametrize("name", list(calls()))
@pytest.mark.parametrize("elsewhere", [0, -1])
def test_a_tensor_on_another_gpu_or_the_host_is_refused(two_gpus, name, elsewhere):  # noqa: F811
    tensors, call = calls()[name]
    for odd in tensors:
        with pytest.raises(ValueError):
            call(**{n: OnGpu(t, elsewhere if n == odd else 1) for n, t in tensors.items()})
    assert name not in [n for n, _ in two_gpus]


@pytest.mark.parametrize("name", list(calls()))
def test_another_type_or_shape_is_refused(two_gpus, name):  # noqa: F811
    """Each tensor in turn as float64, and without its last element or column."""
    tensors, call = calls()[name]
    for odd, t in tensors.items():
        if odd == "workspace":
            continue  # any type of enough bytes
        free = odd in ("table", "ring", "block_lists") or (name, odd) == ("smd_block_trim", "lengths")  # says the sizes
        for bad in (t.double(),) if free else (t.double(), t[..., :-1]):
            with pytest.raises(ValueError):
                call(**{n: OnGpu(bad if n == odd else x, 1) for n, x in tensors.items()})
    assert name not in [n for n, _ in two_gpus]


def test_positions_and_rows_that_do_not_fit_are_refused(two_gpus):  # noqa: F811
    import torch
    t, call = calls()["smd_qk_norm_rope"]
    on = lambda **kw: {n: None if x is None else OnGpu(x, 0) for n, x in {**t, **kw}.items()}  # noqa: E731
    for kw in (dict(positions=None), dict(freqs=None), dict(positions=t["positions"][0]), dict(freqs=t["freqs"][:2]),
               dict(positions=t["positions"].t().contiguous().t()), dict(k=None), dict(q=t["q"].transpose(1, 2))):
        with pytest.raises(ValueError):
            call(**on(**kw))
    call(**on(positions=None, freqs=None))
    call(**on(positions=t["positions"][0], freqs=t["freqs"][0]))
    call(**on(k=None, k_out=None))
    assert [n for n, _ in two_gpus].count("smd_qk_norm_rope") == 3
    t, call = calls()["smd_verify_drafts"]
    with pytest.raises(ValueError):
        call(**{n: OnGpu(x if n != "target" else torch.zeros(3, 5, 10)[:, :4], 0) for n, x in t.items()})
    t, call = calls()["smd_block_trim"]
    for a, b in (("lengths", "new_lengths"), ("state", "new_state")):
        with pytest.raises(ValueError):
            call(**{n: OnGpu(t[a] if n == b else x, 0) for n, x in t.items()})


def test_a_cache_without_bounds_has_no_scores(two_gpus):  # noqa: F811
    tensors, call = calls()["smd_block_scores"]
    with pytest.raises(ValueError):
        call(**{n: None if n == "bounds" else OnGpu(t, 0) for n, t in tensors.items()})
