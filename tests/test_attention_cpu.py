"""The plain statements of the append and of attention, and the host-side
refusals of their entry points: no GPU."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import attention as plain


@pytest.fixture(scope="module")
def misa():
    import importlib.util
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location(
        "_misa_build", os.path.join(root, "long_context_sparse_misa_b200", "build.py"))
    builder = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(builder)
    builder.build()
    import long_context_sparse_misa_b200 as m
    return m


def test_rotation_keeps_lengths_and_adds_angles():
    g = np.random.default_rng(0)
    x = g.standard_normal((3, 8))
    a, b = g.uniform(0, 7, 4), g.uniform(0, 7, 4)
    for il in (False, True):
        y = plain.rotate(x, np.cos(a), np.sin(a), il)
        assert np.allclose((y ** 2).sum(1), (x ** 2).sum(1))
        z = plain.rotate(y, np.cos(b), np.sin(b), il)
        assert np.allclose(z, plain.rotate(x, np.cos(a + b), np.sin(a + b), il))
    # worked: (1, 0) by a quarter turn is (0, 1)
    assert np.allclose(plain.rotate(np.array([[1.0, 5.0, 0.0, 0.0]]), [0.0, 1.0], [1.0, 0.0], False), [[0, 5, 1, 0]])
    assert np.allclose(plain.rotate(np.array([[1.0, 0.0, 5.0, 0.0]]), [0.0, 1.0], [1.0, 0.0], True), [[0, 1, 5, 0]])


def test_attend_closed_forms():
    q, k, v = np.zeros((2, 4)), np.ones((3, 1, 4)), np.arange(12.0).reshape(3, 1, 4)
    out, lse, *_ = plain.attend(q, k, v, 2, [0, 1, 2], 0.5)
    assert np.allclose(out, v.mean(0)) and np.allclose(lse, np.log(3))
    # a bias alone: weights fall by e^-slope a token
    out, lse, *_ = plain.attend(q, k, v, 2, [0, 1, 2], 0.5, slopes=np.array([1.0, 0.0]))
    w = np.exp([-2.0, -1.0, 0.0])
    assert np.allclose(out[0], (w[:, None] * v[:, 0]).sum(0) / w.sum()) and np.isclose(lse[0], np.log(w.sum()))
    # a cap bounds the exponent
    big = plain.attend(np.full((1, 4), 100.0), k, v, 2, [0, 1, 2], 1.0, softcap=3.0)
    assert np.allclose(big[1], 3 + np.log(3))
    none = plain.attend(q, k[:0], v[:0], 2, [], 0.5)
    assert (none[0] == 0).all() and (none[1] == -np.inf).all()


def _problem(misa, **kw):
    d = dict(num_seqs=2, num_queries=4, num_heads=1, head_dim=128, block=64, max_seq_len=1000,
             total_keys=1500, total_blocks=0, key_offsets=8, block_offsets=8, query_offsets=8, q_pos=8)
    d.update(kw)
    return misa._Problem(**d)


def _cache(misa, **kw):
    d = dict(k=256, v=256, dtype=0, num_kv_heads=2, head_dim=128, page_size=16, num_pages=10,
             pages_per_seq=63, page_table=16, page_table_stride=63, page_stride=4096, token_stride=256,
             head_stride=128)
    d.update(kw)
    return misa._KVCache(**d)


OPTS = dict(scale=0.1, softcap=0.0, slopes=None)


def _attention(misa, p=None, c=None, hq=8, opts=None, share=None, out=256, lse=None, ws=256, nb=1 << 30, q=256):
    return misa.lib.misa_attention(ctypes.byref(p or _problem(misa)), ctypes.byref(c or _cache(misa)), q, hq,
                                   ctypes.byref(misa._AttentionOpts(**{**OPTS, **(opts or {})})),
                                   None if share is None else ctypes.byref(misa._SharedPrefix(**share)),
                                   out, lse, ws, nb, None)


def _selected(misa, k=64, idx=16, c=None, hq=8, nb=1 << 30):
    return misa.lib.misa_attention_selected(ctypes.byref(_problem(misa)), ctypes.byref(c or _cache(misa)), 256, hq,
                                            ctypes.byref(misa._AttentionOpts(**OPTS)), idx, k, 256, None, 256, nb, None)


def _append(misa, p=None, c=None, k=256, ks=256, v=256, vs=256, q=None, qs=0, hq=0, q_out=None, rope=None, rows=0, dim=0):
    return misa.lib.misa_cache_append(ctypes.byref(p or _problem(misa)), ctypes.byref(c or _cache(misa)), k, ks, v, vs,
                                      q, qs, hq, q_out, rope, rows, dim, 0, None)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=2), 2), (dict(head_dim=96), 2), (dict(num_kv_heads=0), 1), (dict(num_kv_heads=257), 1),
    (dict(k=None), 1), (dict(k=264), 1), (dict(v=260), 1), (dict(token_stride=100), 1), (dict(head_stride=-8), 1),
    (dict(page_size=0), 1), (dict(page_table=18), 1), (dict(page_table_stride=62), 1), (dict(page_stride=4), 1),
    (dict(num_pages=-1), 1),
])
def test_caches_that_are_refused(misa, change, code):
    c = _cache(misa, **change)
    assert _attention(misa, c=c) == code
    assert _append(misa, c=c) == code
    assert _selected(misa, c=c) == code
    assert misa.lib.misa_attention_workspace_size(ctypes.byref(_problem(misa)), ctypes.byref(c), 8, 0, None) == 0
    assert misa.lib.misa_last_error_string()


@pytest.mark.parametrize("kw,code", [
    (dict(hq=7), 1), (dict(hq=0), 1), (dict(hq=2 * 65), 1), (dict(q=None), 1), (dict(q=264), 1), (dict(out=8), 1),
    (dict(ws=128), 1), (dict(ws=None), 1), (dict(nb=8), 3), (dict(lse=6), 1),
    (dict(opts=dict(softcap=-1.0)), 1), (dict(opts=dict(softcap=float("nan"))), 1),
    (dict(opts=dict(scale=float("inf"))), 1), (dict(opts=dict(slopes=6)), 1),
    (dict(share=dict(num_groups=-1, max_len=5, seq_offsets=8, lens=8)), 1),
    (dict(share=dict(num_groups=1, max_len=1001, seq_offsets=8, lens=8)), 1),
    (dict(share=dict(num_groups=1, max_len=5, seq_offsets=None, lens=8)), 1),
    (dict(share=dict(num_groups=1, max_len=5, seq_offsets=8, lens=6)), 1),
])
def test_attention_calls_that_are_refused(misa, kw, code):
    assert _attention(misa, **kw) == code


def test_selected_calls_that_are_refused(misa):
    assert _selected(misa, k=0) == 1 and _selected(misa, k=65537) == 1
    assert _selected(misa, idx=None) == 1 and _selected(misa, idx=18) == 1
    assert _selected(misa, nb=8) == 3
    size = misa.lib.misa_attention_workspace_size
    p, c = _problem(misa), _cache(misa)
    share = misa._SharedPrefix(num_groups=1, max_len=5, seq_offsets=8, lens=8)
    assert size(ctypes.byref(p), ctypes.byref(c), 8, 64, ctypes.byref(share)) == 0
    assert size(ctypes.byref(p), ctypes.byref(c), 8, -1, None) == 0
    assert size(ctypes.byref(p), ctypes.byref(c), 8, 64, None) > 0


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(k=264), dict(ks=248), dict(ks=257), dict(v=None), dict(v=8), dict(vs=128), dict(q=256, qs=1024, hq=8),
    dict(q=256, qs=512, hq=8, q_out=512), dict(q=256, qs=1024, hq=0, q_out=512), dict(q=256, qs=2048, hq=8, q_out=256),
    dict(q_out=256), dict(rope=8, rows=10, dim=64), dict(rope=256, rows=0, dim=64), dict(rope=256, rows=10, dim=24),
    dict(rope=256, rows=10, dim=256), dict(rope=256, rows=10, dim=0),
])
def test_append_calls_that_are_refused(misa, kw):
    assert _append(misa, **kw) == 1
    assert _append(misa, c=_cache(misa, v=None)) == 1                      # values without a place


def test_batches_that_are_refused(misa):
    for bad in (dict(num_seqs=0), dict(num_queries=-1), dict(max_seq_len=0), dict(key_offsets=None), dict(query_offsets=None),
                dict(q_pos=None), dict(total_keys=-1)):
        assert _attention(misa, p=_problem(misa, **bad)) == 1
        assert _append(misa, p=_problem(misa, **bad)) == 1
    # no queries: nothing to do, whatever the indexer's fields hold
    none = _problem(misa, num_queries=0, q_pos=None, num_heads=0, head_dim=0, block=0, block_offsets=None)
    assert _attention(misa, p=none) == 0 and _append(misa, p=none) == 0


def test_python_checks_name_what_is_wrong(misa):
    cpu = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        misa.KVCache(cpu)
    with pytest.raises(ValueError, match="non-decreasing"):
        misa.SharedPrefix([0, 2, 1], [3, 4], device="cpu")
    with pytest.raises(ValueError, match="non-decreasing"):
        misa.SharedPrefix([0, 2], [-3], device="cpu")
    t = misa.rope_table(3, 4, theta=100.0, device="cpu")
    want = [[1, 1, 0, 0], [np.cos(1), np.cos(0.1), np.sin(1), np.sin(0.1)], [np.cos(2), np.cos(0.2), np.sin(2), np.sin(0.2)]]
    assert np.allclose(t.numpy(), want, atol=1e-7)
