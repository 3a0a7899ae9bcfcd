"""The paged-cache calls without a GPU: the oracle against closed forms, and
the refusals that come before any launch."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

from oracle import paged as opaged
from sparse_mla_decode_gb300 import binding as smd

A = 1 << 20  # an aligned address that nothing is read from


def test_e4m3_codes():
    v = opaged.VALUES
    assert v[0x7e] == 448 and v[0x08] == 2.0 ** -6 and v[0x01] == 2.0 ** -9 and np.isnan(v[0x7f])
    finite = np.array([c for c in range(256) if (c & 127) != 127])
    assert np.array_equal(opaged.e4m3_encode(v[finite]), finite)
    # halfway values go to the even code; the rest to the nearer one
    mid = (v[:126] + v[1:127]) / 2
    even = np.arange(126) + (np.arange(126) % 2)
    assert np.array_equal(opaged.e4m3_encode(mid), even)
    assert np.array_equal(opaged.e4m3_encode(np.nextafter(mid, 0)), np.arange(126))
    assert opaged.e4m3_encode(np.array([1e9]))[0] == 0x7e


def test_power_is_the_least_that_fits():
    for a in (448.0, 449.0, 447.9, 1.0, 1.75, 1.7500001, 2.0 ** -100, 3e38, 896.0, 897.0):
        s = opaged.power(a)
        assert a / s <= 448 and (a / (s / 2) > 448 or s == 2.0 ** -120)
    assert opaged.power(0.0) == 2.0 ** -120 and opaged.power(1e-38) == 2.0 ** -120


def test_decode_of_equal_logits_is_the_mean_and_of_one_token_its_value():
    rng = np.random.default_rng(0)
    codes = [opaged.e4m3_encode(rng.standard_normal((3, 1, 16, 64)) * 50) for _ in "kv"]
    scales = [np.full((3, 1), 0.5), np.full((3, 1), 0.25)]
    v = opaged.VALUES[codes[1]] * 0.25
    table = np.array([[2, 0], [1, 1]])
    out, lse, _, _ = opaged.paged_decode(np.zeros((2, 1, 64)), codes, scales, table, [20, 1], 0.1)
    rows = np.concatenate([v[2, 0], v[0, 0, :4]])
    assert np.allclose(out[0, 0], rows.mean(0)) and np.isclose(lse[0, 0], np.log(20))
    assert np.allclose(out[1, 0], v[1, 0, 0]) and lse[1, 0] == 0.0
    out, lse, _, _ = opaged.paged_decode(np.zeros((2, 1, 64)), codes, scales, table, [0, 0], 0.1)
    assert (out == 0).all() and np.isneginf(lse).all()


def test_scores_bound_the_products():
    rng = np.random.default_rng(1)
    k = opaged.bf16_round(rng.standard_normal((40, 2, 64)))
    pools = [np.zeros((3, 2, 16, 64), dtype=np.uint8) for _ in "kv"]
    bounds = np.zeros((3, 2, 2, 64))
    opaged.paged_append(pools, [np.zeros((3, 2)) for _ in "kv"], bounds, [k, k], np.arange(40))
    q = rng.standard_normal((1, 6, 64))
    s = opaged.block_scores(q, bounds, np.array([[0, 1, 2, 0]]), [40], 16, 1)
    assert np.isnan(s[0, :, 3]).all()
    for h in range(2):
        dots = k[:, h] @ q[0, 3 * h:3 * h + 3].T
        for j in range(3):
            assert dots[16 * j:16 * j + 16].max() <= s[0, h, j] + 1e-9


def cache(**kw):
    c = smd.SmdPagedCache()
    f = dict(bounds=A, pages=10, heads=2, page_size=32, head_dim=128)
    f.update(kw)
    for name, v in f.items():
        setattr(c, name, (ctypes.c_int64 * 3)(*v) if name.endswith("stride") else v)
    return c


def init(**kw):
    return smd.lib().smd_paged_cache_init(ctypes.byref(cache(**kw)))


KV = dict(k=A, v=A, k_scale=A, v_scale=A, k_stride=(8192, 4096, 128), v_stride=(8192, 4096, 128))


@pytest.mark.parametrize("kw,code", [
    ({}, smd.SMD_OK), (dict(bounds=0), smd.SMD_ERR_NULL), (dict(k=A), smd.SMD_ERR_NULL),
    (dict(v=A), smd.SMD_ERR_NULL), (dict(KV, k_scale=0), smd.SMD_ERR_NULL),
    (dict(pages=0), smd.SMD_ERR_SHAPE), (dict(heads=0), smd.SMD_ERR_SHAPE),
    (dict(page_size=8), smd.SMD_ERR_SHAPE), (dict(page_size=40), smd.SMD_ERR_SHAPE),
    (dict(page_size=272), smd.SMD_ERR_SHAPE), (dict(head_dim=96), smd.SMD_ERR_SHAPE),
    (dict(pages=2 ** 26), smd.SMD_ERR_SHAPE), (dict(bounds=A + 8), smd.SMD_ERR_ALIGN),
    (dict(KV, k_scale=A + 2), smd.SMD_ERR_ALIGN), (dict(KV, k=A + 8), smd.SMD_ERR_ALIGN),
    (dict(KV, k_stride=(8192, 4096, 120)), smd.SMD_ERR_SHAPE),
    (dict(KV, v_stride=(-8192, 4096, 128)), smd.SMD_ERR_SHAPE),
    (dict(KV, v_stride=(8192, 4096, 136)), smd.SMD_ERR_ALIGN)])
def test_cache_description(kw, code):
    assert init(**kw) == code


def test_a_null_or_unfinished_cache_is_refused():
    so, c = smd.lib(), cache()
    assert so.smd_paged_cache_init(None) == smd.SMD_ERR_NULL
    assert so.smd_paged_workspace_bytes(None) == smd.SMD_ERR_NULL
    assert so.smd_paged_workspace_bytes(ctypes.byref(c)) == smd.SMD_ERR_PLAN
    assert so.smd_paged_append(ctypes.byref(c), A, 256, A, 256, A, 1, 0) == smd.SMD_ERR_PLAN
    assert so.smd_paged_append(None, A, 256, A, 256, A, 1, 0) == smd.SMD_ERR_NULL
    assert init_rows(c) == smd.SMD_ERR_PLAN


def init_rows(c, q=A, q_stride=512, table=A, table_stride=4, width=4, lengths=A, R=2, G=1, Hq=4,
              first=0, last=0, scores=A, score_stride=4):
    return smd.lib().smd_block_scores(q, q_stride, ctypes.byref(c), table, table_stride, width,
                                      lengths, R, G, Hq, first, last, scores, score_stride, 0)


@pytest.mark.parametrize("kw,code", [
    (dict(R=0), smd.SMD_OK), (dict(R=-1), smd.SMD_ERR_SHAPE), (dict(G=0), smd.SMD_ERR_SHAPE),
    (dict(G=9), smd.SMD_ERR_SHAPE), (dict(Hq=3), smd.SMD_ERR_SHAPE), (dict(Hq=0), smd.SMD_ERR_SHAPE),
    (dict(Hq=258), smd.SMD_ERR_SHAPE), (dict(width=0), smd.SMD_ERR_SHAPE),
    (dict(table_stride=3), smd.SMD_ERR_SHAPE), (dict(width=2 ** 27, table_stride=2 ** 27), smd.SMD_ERR_SHAPE),
    (dict(q_stride=511), smd.SMD_ERR_SHAPE), (dict(q_stride=516), smd.SMD_ERR_SHAPE),
    (dict(R=2 ** 30), smd.SMD_ERR_SHAPE), (dict(q=0), smd.SMD_ERR_NULL),
    (dict(table=0), smd.SMD_ERR_NULL), (dict(lengths=0), smd.SMD_ERR_NULL),
    (dict(scores=0), smd.SMD_ERR_NULL), (dict(q=A + 8), smd.SMD_ERR_ALIGN),
    (dict(table=A + 2), smd.SMD_ERR_ALIGN), (dict(scores=A + 1), smd.SMD_ERR_ALIGN),
    (dict(first=-1), smd.SMD_ERR_SHAPE), (dict(last=-1), smd.SMD_ERR_SHAPE),
    (dict(score_stride=3), smd.SMD_ERR_SHAPE)])
def test_rows_of_queries(kw, code):
    c = cache()
    assert smd.lib().smd_paged_cache_init(ctypes.byref(c)) == smd.SMD_OK
    assert init_rows(c, **kw) == code


def test_the_decode_and_the_append_want_keys_and_values():
    c = cache()
    assert smd.lib().smd_paged_cache_init(ctypes.byref(c)) == smd.SMD_OK
    assert smd.lib().smd_paged_decode(A, 512, ctypes.byref(c), A, 4, 4, A, 2, 1, 4, 0.1, None, None, 0,
                                      A, A, None, A, 1 << 30, 0) == smd.SMD_ERR_NULL
    assert smd.lib().smd_paged_append(ctypes.byref(c), A, 256, A, 256, A, 1, 0) == smd.SMD_ERR_NULL


@pytest.mark.parametrize("kw,code", [
    (dict(R=-1), smd.SMD_ERR_SHAPE), (dict(R=8193), smd.SMD_ERR_SHAPE), (dict(T=-1), smd.SMD_ERR_SHAPE),
    (dict(pages=0), smd.SMD_ERR_SHAPE), (dict(P=0), smd.SMD_ERR_SHAPE), (dict(width=0), smd.SMD_ERR_SHAPE),
    (dict(stride=3), smd.SMD_ERR_SHAPE), (dict(pages=2 ** 30, P=2), smd.SMD_ERR_SHAPE),
    (dict(width=2 ** 28, stride=2 ** 28), smd.SMD_ERR_SHAPE), (dict(lengths=0), smd.SMD_ERR_NULL),
    (dict(new=0), smd.SMD_ERR_NULL), (dict(table=0), smd.SMD_ERR_NULL), (dict(ring=0), smd.SMD_ERR_NULL),
    (dict(state=0), smd.SMD_ERR_NULL), (dict(new_lengths=0), smd.SMD_ERR_NULL),
    (dict(new_state=0), smd.SMD_ERR_NULL), (dict(starts=0), smd.SMD_ERR_NULL),
    (dict(slots=0), smd.SMD_ERR_NULL), (dict(lengths=A + 2), smd.SMD_ERR_ALIGN),
    (dict(state=A + 4), smd.SMD_ERR_ALIGN), (dict(positions=A + 1), smd.SMD_ERR_ALIGN)])
def test_tables(kw, code):
    f = dict(lengths=A, new=A, R=2, table=A, stride=4, width=4, ring=A, pages=8, state=A, P=16, T=4,
             new_lengths=A, new_state=A, starts=A, slots=A, positions=0, status=0)
    f.update(kw)
    assert smd.lib().smd_block_tables(*f.values(), 0) == code


def test_the_new_status_has_a_text():
    assert smd.smd_status_str(smd.SMD_ERR_PAGES) != "unknown status"


class OnGpu:
    """A host tensor that says it is on a GPU."""

    def __init__(self, t, index):
        self.t, self.index, self.device, self.is_cuda = t, index, f"cuda:{index}", index >= 0

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.index


@pytest.fixture
def two_gpus(monkeypatch):
    """The library's calls, recorded with the GPU that is current at each."""
    import torch
    now, calls = [0], []

    class Library:
        def __getattr__(self, name):
            def call(*args):
                calls.append((name, now[0]))
                return 16 if name == "smd_paged_workspace_bytes" else smd.SMD_OK
            return call

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *_):
            now[0] = self.before

    monkeypatch.setattr(smd, "lib", Library)
    monkeypatch.setattr(smd, "_so", Library)
    monkeypatch.setattr(smd, "_current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    return calls


def paged_calls():
    """Each call's tensors by name, and the call on them."""
    import torch

    def zeros(*shape, dtype=torch.int32):
        return torch.zeros(shape, dtype=dtype)

    bf, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    cache = dict(k=zeros(4, 2, 16, 64, dtype=u8), v=zeros(4, 2, 16, 64, dtype=u8), k_scale=zeros(4, 2, dtype=f32),
                 v_scale=zeros(4, 2, dtype=f32), bounds=zeros(4, 2, 2, 64, dtype=bf))
    rows = dict(q=zeros(3, 4, 64, dtype=bf), table=zeros(3, 2), lengths=zeros(3))

    def on_cache(call):
        def with_cache(**t):
            c = smd.PagedCache(**{n: t.pop(n) for n in cache})
            call(c, t)
        return with_cache

    return {
        "smd_block_tables": (dict(lengths=zeros(3), new_tokens=zeros(3), table=zeros(3, 2), ring=zeros(4),
                                  state=zeros(2, dtype=torch.int64), new_lengths=zeros(3),
                                  new_state=zeros(2, dtype=torch.int64), starts=zeros(4), slots=zeros(5),
                                  positions=zeros(5), status=zeros(1)),
                             lambda **t: smd.block_tables(page_size=16, stream=7, **t)),
        "smd_paged_append": (dict(cache, k_new=zeros(5, 2, 64, dtype=bf), v_new=zeros(5, 2, 64, dtype=bf),
                                  slots=zeros(5)),
                             on_cache(lambda c, t: smd.paged_append(c, t["k_new"], t["v_new"], t["slots"], stream=7))),
        "smd_block_scores": (dict(cache, **rows, out=zeros(3, 2, 2, dtype=bf)),
                             on_cache(lambda c, t: smd.block_scores(cache=c, stream=7, **t))),
        "smd_paged_decode": (dict(cache, **rows, block_lists=zeros(3, 2, 1), block_counts=zeros(3, 2),
                                  out=zeros(3, 4, 64, dtype=bf), lse=zeros(3, 4, dtype=f32),
                                  status=zeros(1), workspace=zeros(16, dtype=u8)),
                             on_cache(lambda c, t: smd.paged_decode(cache=c, sm_scale=0.1, stream=7, **t)))}


CALLS = ["smd_block_tables", "smd_paged_append", "smd_block_scores", "smd_paged_decode"]


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("index", [0, 1])
def test_a_call_runs_on_the_gpu_of_its_tensors(two_gpus, name, index):
    tensors, call = paged_calls()[name]
    call(**{n: OnGpu(t, index) for n, t in tensors.items()})
    assert (name, index) in two_gpus
    if name == "smd_paged_decode":
        cache = smd.PagedCache(bounds=OnGpu(tensors["bounds"], index), page_size=16)
        assert smd.paged_workspace_bytes(cache) == 16
        assert two_gpus[-1] == ("smd_paged_workspace_bytes", index)


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("elsewhere", [0, -1])
def test_a_tensor_on_another_gpu_or_the_host_is_refused(two_gpus, name, elsewhere):
    tensors, call = paged_calls()[name]
    for odd in tensors:
        with pytest.raises(ValueError):
            call(**{n: OnGpu(t, elsewhere if n == odd else 1) for n, t in tensors.items()})
    assert name not in [n for n, _ in two_gpus]


@pytest.mark.parametrize("name", ["smd_block_tables", "smd_paged_decode"])
def test_the_status_word_is_checked(two_gpus, name):
    tensors, call = paged_calls()[name]
    for status in (tensors["status"][:0], tensors["status"].long(), tensors["status"].float()):
        with pytest.raises(ValueError):
            call(**{n: OnGpu(t, 1) for n, t in dict(tensors, status=status).items()})
    assert name not in [n for n, _ in two_gpus]


@pytest.mark.parametrize("option,value", [("--requests", 0), ("--requests", 8193), ("--context", 0), ("--steps", 0),
                                          ("--steps", -2), ("--pages", 0)])
def test_the_step_command_refuses_sizes_that_it_cannot_run(option, value, capsys):
    from sparse_mla_decode_gb300 import paged_step
    with pytest.raises(SystemExit) as e:
        paged_step.main([option, str(value)])
    assert e.value.code == 2 and option in capsys.readouterr().err


def test_scores_of_one_head_go_to_rows_of_any_spacing(two_gpus):
    """A dimension of one head has whatever stride the caller's view gave it."""
    import torch
    tensors, call = paged_calls()["smd_block_scores"]
    one = {n: t[:, :1].contiguous() if n in ("k", "v", "k_scale", "v_scale", "bounds") else t
           for n, t in tensors.items()}
    wide = torch.zeros((3, 9), dtype=torch.bfloat16)
    for out in (wide[:, None, :2], wide[:, :2][:, None], wide.as_strided((3, 1, 2), (9, 100, 1))):
        call(**{n: OnGpu(t, 0) for n, t in dict(one, out=out).items()})
    assert [n for n, _ in two_gpus].count("smd_block_scores") == 3
    two = dict(tensors, out=torch.zeros((3, 5, 2), dtype=torch.bfloat16)[:, :2])
    with pytest.raises(ValueError):
        call(**{n: OnGpu(t, 0) for n, t in two.items()})
