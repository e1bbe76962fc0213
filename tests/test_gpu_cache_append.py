"""cache_append on a B200 against the definition in 64 bits: every row it
writes within the rounding of its type, every other row bit for bit as before."""
import numpy as np
import pytest
import torch

import long_context_sparse_misa_b200 as misa
from oracle import attention as plain
from tests.attention_cases import HALF_STEP, Batch, assert_status_ok

pytestmark = pytest.mark.gpu


def _run(b, rotated, interleaved, with_q, fused, seed=1, values=True):
    g = torch.Generator().manual_seed(seed)
    r, hkv, hq, d = b.rows, b.hkv, b.hq if with_q else 0, b.dim
    heads = hq + hkv * (2 if values else 1)
    x = torch.randn(r, heads, d, generator=g).to(b.dtype)
    dev = x.cuda()
    part = lambda lo, n: dev[:, lo:lo + n] if fused else dev[:, lo:lo + n].contiguous()
    q = part(0, hq) if with_q else None
    q_out = torch.full((r, hq, d), 9.0, dtype=b.dtype, device="cuda") if with_q else None
    rope = misa.rope_table(max(b.lens) + 5, rotated) if rotated else None
    cache = b.cache if values else misa.KVCache(b.k, None, getattr(b, "table_dev", None))
    before_k, before_v = b.k.clone(), b.v.clone()
    misa.cache_append(b.prob, cache, part(hq, hkv), part(hq + hkv, hkv) if values else None, q=q,
                      q_out=q_out, rope=rope, interleaved=interleaved)
    return x, rope, q_out, before_k, before_v


def _check(b, x, rope, q_out, before_k, before_v, interleaved, values=True):
    hkv, hq = b.hkv, 0 if q_out is None else b.hq
    u = HALF_STEP[b.dtype]
    k, v = b.k.cpu(), b.v.cpu()
    want_k, want_v = before_k.cpu().clone(), before_v.cpu().clone()
    seen = torch.zeros(k.shape[:-2], dtype=torch.bool)
    ko = np.concatenate([[0], np.cumsum(b.lens)])

    def near(got, raw, p, what):
        f = raw.float().numpy().astype(np.float64)
        n = 0 if rope is None else rope.shape[1]
        want = f
        if n:
            row = rope[p].cpu().numpy().astype(np.float64)
            want = f.copy()
            want[:, :n] = plain.rotate(f[:, :n], row[:n // 2], row[n // 2:], interleaved)
            assert torch.equal(got[:, n:], raw[:, n:]), what
        else:
            assert torch.equal(got, raw), what
        # one rounding to the type, on fp32 products and one fp32 sum of values up to max|x|
        tol = u * np.abs(want) * (1 + u) + 2.0 ** -21 * np.abs(f).max() + 2.0 ** -25
        assert (np.abs(got.float().numpy() - want) <= tol).all(), what

    for t in range(b.T):
        s, p = b.seq[t], b.pos[t]
        at = (ko[s] + p,) if b.table is None else (int(b.table[s, p // b.page]), p % b.page)
        near(k[at], x[t, hq:hq + hkv], p, f"k of token {t}")
        if values:
            assert torch.equal(v[at], x[t, hq + hkv:]), f"v of token {t}"
            want_v[at] = v[at]
        want_k[at] = k[at]
        seen[at] = True
        if hq:
            near(q_out[t].cpu(), x[t, :hq], p, f"q of token {t}")
    bits = lambda c: c.contiguous().view(torch.int16)
    assert torch.equal(bits(k), bits(want_k)) and torch.equal(bits(v), bits(want_v)), "another row changed"
    if hq:
        assert (q_out[b.T:] == 9).all(), "padding rows were written"


SHAPES = [  # lens, queries, hq, hkv, dim, page, heads_first, packed, pad
    ([40], [[39]], 8, 2, 128, 16, False, False, 0),
    ([1], [[0]], 1, 1, 64, 1, False, False, 0),
    ([100, 7, 0, 33], [[97, 98, 99], [6], [], [0, 32]], 6, 3, 64, 7, True, False, 3),
    ([300, 2], [list(range(300)), [1]], 4, 4, 128, 64, True, False, 1),
    ([50, 60], [[49], [10, 59]], 16, 8, 128, 16, False, True, 0),
]


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rotated,interleaved,with_q,fused",
                         [(1.0, False, True, True), (0.5, True, True, False), (1.0, True, False, True),
                          (0, False, True, True), (0.5, False, True, True)])
def test_append_matches_the_definition(shape, dtype, rotated, interleaved, with_q, fused):
    lens, qs, hq, hkv, dim, page, hf, packed, pad = SHAPES[shape]
    b = Batch(lens, qs, hq, hkv, dim, page, dtype, seed=shape, heads_first=hf, packed=packed, pad_rows=pad)
    got = _run(b, int(rotated * dim), interleaved, with_q, fused)
    assert_status_ok()
    _check(b, *got, interleaved)


def test_append_keys_only_and_rotation_in_place():
    b = Batch([70, 30], [[69], [28, 29]], 4, 1, packed=True)
    got = _run(b, 128, False, False, False, values=False)
    assert_status_ok()
    _check(b, *got, False, values=False)
    q = b.q.clone()
    rope = misa.rope_table(70, 128)
    out = torch.empty_like(q)
    new = torch.randn(b.T, 1, 128, device="cuda").to(b.dtype)
    misa.cache_append(b.prob, b.cache, new, new, q=q, q_out=out, rope=rope)
    misa.cache_append(b.prob, b.cache, new, new, q=q, q_out=q, rope=rope)
    assert_status_ok()
    assert torch.equal(q, out)


def test_append_many_sequences_and_far_positions():
    # 1500 sequences (three rounds of the search), some without a token, one far position
    lens = [5 + s % 9 for s in range(1500)]
    lens[700] = 200_000
    qs = [[n - 1] if s % 3 else [] for s, n in enumerate(lens)]
    qs[700] = [199_998, 199_999]
    b = Batch(lens, qs, 2, 1, dim=64, page=16, seed=4)
    got = _run(b, 64, False, True, True)
    assert_status_ok()
    _check(b, *got, False)


def test_append_flags_and_skips_what_has_no_place():
    b = Batch([40, 40, 40], [[3], [39], [5]], 2, 1, page=16)
    b.prob.q_pos.copy_(torch.tensor([40, 39, -1], dtype=torch.int32))      # two outside their sequences
    bad = b.table.copy()
    bad[1, 2] = 1000                                                        # a page that is not there
    b.table_dev.copy_(torch.from_numpy(bad))
    before = b.k.clone(), b.v.clone()
    x = torch.ones(3, 1, 128, device="cuda", dtype=b.dtype)
    q_out = torch.full((3, 2, 128), 9.0, device="cuda", dtype=b.dtype)
    misa.cache_append(b.prob, b.cache, x, x, q=b.q, q_out=q_out)
    code, bits = misa.stream_status()
    assert bits == 0x2 | 0x4
    same = lambda a, c: torch.equal(a.view(torch.int16), c.view(torch.int16))
    assert same(b.k, before[0]) and same(b.v, before[1]) and (q_out == 9).all()
    # a position past the rotation's table
    b = Batch([40], [[39]], 2, 1, page=16)
    before = b.k.clone()
    misa.cache_append(b.prob, b.cache, x[:1], x[:1], rope=misa.rope_table(39, 128))
    assert misa.stream_status()[1] == 0x2 and same(b.k, before)


def test_append_carries_infinities_and_nan():
    b = Batch([20], [[19]], 2, 1)
    x = torch.zeros(1, 1, 128, device="cuda", dtype=b.dtype)
    x[0, 0, 3], x[0, 0, 100] = float("inf"), float("nan")
    misa.cache_append(b.prob, b.cache, x, x)
    assert_status_ok()
    at = int(b.table[0, 1]), 3
    assert b.v[at][0, 3].isinf() and b.v[at][0, 100].isnan() and b.k[at][0, 3].isinf()
