"""attention and attention_selected on a B200 against the definition in 64
bits: every element of every row within the bound of its roundings."""
import numpy as np
import pytest
import torch

import long_context_sparse_misa_b200 as misa
from tests.attention_cases import Batch, assert_status_ok

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


def _last(lens, n):
    return [list(range(max(0, L - n), L)) for L in lens]


def _slopes(hq):
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / hq) for i in range(hq)], device="cuda")


WHOLE = [  # lens, queries, hq, hkv, dim, page, dtype, layout
    ([1], [[0]], 1, 1, 128, 16, BF, {}),
    ([1], [[0]], 4, 2, 64, 1, FP, {}),
    ([2, 31, 32, 33], _last([2, 31, 32, 33], 1), 8, 1, 128, 16, BF, {}),
    ([127, 128, 129, 300], _last([127, 128, 129, 300], 2), 6, 2, 128, 33, FP, dict(heads_first=True)),
    ([1000, 0, 17], [[999], [], [0, 5, 16]], 16, 2, 64, 64, BF, dict(pad_rows=2)),
    ([513, 90], _last([513, 90], 3), 7, 1, 128, 100, BF, dict(packed=True)),
    ([2500], _last([2500], 1), 32, 4, 128, 16, FP, {}),
    ([700], _last([700], 1), 64, 1, 64, 16, BF, {}),
    ([260, 100], _last([260, 100], 20), 10, 2, 128, 16, BF, {}),
    ([300, 500], [list(range(300)), list(range(100, 400))], 2, 1, 128, 48, BF, dict(heads_first=True)),
    ([400], [list(range(400))], 4, 2, 64, 16, FP, {}),
    # long keys for few rows: cut into equal parts over all blocks
    ([20000], [[19999]], 4, 1, 128, 64, BF, {}),
    ([9000, 0, 3, 15001, 128], [[8998, 8999], [], [2], [15000, 7], [127]], 6, 2, 64, 33, FP, dict(pad_rows=1)),
    ([7000] * 3 + [1, 5000], _last([7000] * 3 + [1, 5000], 2), 24, 1, 128, 16, BF, dict(packed=True)),
    ([12000], [[3, 700, 11999]], 36, 1, 64, 16, BF, dict(heads_first=True)),
]


@pytest.mark.parametrize("case", range(len(WHOLE)))
@pytest.mark.parametrize("softcap,bias", [(0.0, False), (5.0, False), (0.0, True), (30.0, True)])
def test_attention_matches_the_definition(case, softcap, bias):
    lens, qs, hq, hkv, dim, page, dt, kw = WHOLE[case]
    b = Batch(lens, qs, hq, hkv, dim, page, dt, seed=case, **kw)
    opts = dict(softcap=softcap, slopes=_slopes(hq) if bias else None)
    out, lse = b.attention(**opts)
    assert_status_ok()
    b.check(out, lse, **opts)


SHARED = [  # lens, queries per sequence, groups {first: (end, length)}, hq, hkv, dim, page, dtype
    ([140, 150, 133], 1, {0: (3, 128)}, 8, 2, 128, 16, BF),
    ([40, 41], 2, {0: (2, 37)}, 4, 1, 64, 16, FP),                       # ends inside a page
    ([700, 650, 90, 640, 645], 1, {0: (2, 600), 3: (5, 639)}, 16, 2, 128, 64, BF),   # one in no group
    ([300] * 40, 1, {0: (40, 256)}, 8, 1, 128, 16, BF),                  # 320 rows on one key head
    ([1300] * 9, 3, {0: (9, 1290)}, 32, 2, 64, 33, BF),
    ([50, 60], 1, {0: (2, 50)}, 2, 1, 128, 16, BF),                      # nothing of its own in the first
    ([50, 60, 70], 1, {0: (2, 0), 2: (3, 60)}, 2, 1, 128, 16, BF),       # an empty prefix, a group of one
    ([9000, 9500, 900, 20000], 1, {0: (3, 640)}, 4, 1, 128, 64, BF),     # long ones of their own behind it
    ([5000] * 6 + [400], 2, {0: (3, 4096), 3: (7, 300)}, 16, 2, 64, 16, FP),
]


@pytest.mark.parametrize("case", range(len(SHARED)))
@pytest.mark.parametrize("softcap,bias", [(0.0, False), (10.0, True)])
def test_shared_prefix_matches_the_definition(case, softcap, bias):
    lens, n, groups, hq, hkv, dim, page, dt = SHARED[case]
    b = Batch(lens, _last(lens, n), hq, hkv, dim, page, dt, seed=case, prefix=groups)
    # offsets with the sequences between groups as groups of no length
    so, ln, at = [0], [], 0
    for a, (e, length) in sorted(groups.items()):
        if a > at:
            so.append(a)
            ln.append(0)
        so.append(e)
        ln.append(length)
        at = e
    share = misa.SharedPrefix(so, ln)
    opts = dict(softcap=softcap, slopes=_slopes(hq) if bias else None)
    out, lse = b.attention(share=share, **opts)
    assert_status_ok()
    b.check(out, lse, **opts)
    # the prefix is read where the first sequence of its group keeps it: the others' pages there do not matter
    if page == 16 and not any(length % page for _, length in groups.values()):
        table = b.table.copy()
        for a, (e, length) in groups.items():
            table[a + 1:e, :length // page] = -1
        b.table_dev.copy_(torch.from_numpy(table))
        again, lse2 = b.attention(share=share, **opts)
        assert_status_ok()
        assert torch.equal(out, again) and torch.equal(lse, lse2)


def _lists(b, k, seed, full=False):
    g = np.random.default_rng(seed)
    idx = np.full((b.rows, k), -1, np.int32)
    for t in range(b.T):
        n = b.pos[t] + 1
        m = min(k, n) if full else int(g.integers(0, min(k, n) + 1))
        idx[t, g.permutation(k)[:m]] = g.choice(n, m, replace=False)
    return idx


SELECTED = [  # lens, queries per sequence, k, hq, hkv, dim, page, dtype
    ([1], 1, 1, 1, 1, 128, 16, BF),
    ([100, 40], 2, 16, 4, 2, 64, 16, FP),
    ([500, 3, 260], 1, 200, 8, 1, 128, 33, BF),
    ([4000], 3, 2048, 32, 2, 128, 64, BF),
    ([900], 40, 300, 64, 1, 128, 16, BF),
    ([900, 300], 9, 129, 20, 1, 64, 100, FP),
    ([600], 5, 77, 48, 1, 128, 16, FP),
]


@pytest.mark.parametrize("case", range(len(SELECTED)))
@pytest.mark.parametrize("softcap,bias", [(0.0, False), (20.0, True)])
def test_selected_matches_the_definition(case, softcap, bias):
    lens, n, k, hq, hkv, dim, page, dt = SELECTED[case]
    b = Batch(lens, _last(lens, n), hq, hkv, dim, page, dt, seed=case, pad_rows=case % 2)
    idx = _lists(b, k, case, full=case == 3)
    idx[0] = -1                                          # a row that selects nothing
    opts = dict(softcap=softcap, slopes=_slopes(hq) if bias else None)
    out, lse = b.selected(idx, **opts)
    assert_status_ok()
    b.check(out, lse, idx=idx, **opts)


def test_selecting_everything_is_attention():
    b = Batch([300, 200], _last([300, 200], 2), 8, 2, 128, 16, BF)
    g = np.random.default_rng(0)
    idx = np.full((b.T, 320), -1, np.int32)
    for t in range(b.T):
        idx[t, g.permutation(320)[:b.pos[t] + 1]] = np.arange(b.pos[t] + 1)
    out, lse = b.selected(idx)
    b.check(out, lse)


def test_lists_count_repeats_and_flag_what_lies_ahead():
    b = Batch([100], [[50, 99]], 4, 1)
    idx = np.array([[3, 3, 3, 9, -1], [1, 2, 98, 99, 0]], np.int32)
    out, lse = b.selected(idx)
    assert_status_ok()
    b.check(out, lse, idx=idx)
    idx[0, 3] = 51                                       # behind its query: skipped
    out, lse = b.selected(idx)
    assert misa.stream_status()[1] == 0x4
    b.check(out, lse, idx=idx)


def test_bad_positions_and_pages_are_flagged_and_give_zeros():
    b = Batch([100, 80, 60], _last([100, 80, 60], 1), 4, 2, page=16)
    b.prob.q_pos[1] = 80
    out, lse = b.attention()
    assert misa.stream_status()[1] == 0x4
    assert (out[1] == 0).all() and (lse[1] == -float("inf")).all()
    b.check(out, lse, rows=[0, 2])
    b.prob.q_pos[1] = 79
    b.table_dev[2, 1] = 1 << 20                          # tokens 16..31 have no row: as if masked
    out, lse = b.attention()
    assert misa.stream_status()[1] == 0x2
    idx = np.full((3, 60), -1, np.int32)
    idx[2, :44] = [p for p in range(60) if not 16 <= p < 32]
    b.check(out, lse, rows=[0, 1])
    b.check(out, lse, idx=idx, rows=[2])


def test_what_later_tokens_hold_reaches_no_earlier_query():
    # chunks of several queries: a query must not see infinities or NaN of tokens behind it
    for hq, n in ((2, 3), (16, 3), (4, 150)):
        b = Batch([400, 333], _last([400, 333], n), hq, 1, page=16)
        clean, lse = b.attention()
        for s, L in enumerate(b.lens):
            for p, bad in ((L - 1, float("nan")), (L - 2, float("inf"))):
                at = int(b.table[s, p // 16]), p % 16
                b.k[at], b.v[at] = bad, bad
        out, lse2 = b.attention()
        assert_status_ok()
        early = [t for t in range(b.T) if b.pos[t] < b.lens[b.seq[t]] - 2]
        assert torch.equal(out[early], clean[early]) and torch.equal(lse[early], lse2[early])
        late = [t for t in range(b.T) if b.pos[t] == b.lens[b.seq[t]] - 1]
        assert out[late].isnan().all()


@pytest.mark.parametrize("hq,n,dt", [(2, 3, BF), (16, 3, FP), (32, 2, BF), (4, 150, BF), (4, 150, FP), (48, 1, BF)])
def test_an_infinite_value_reaches_the_queries_that_see_it(hq, n, dt):
    b = Batch([400, 333], _last([400, 333], n), hq, 1, page=16, dtype=dt)
    clean, lse = b.attention()
    for s, L in enumerate(b.lens):
        for p, d, bad in ((L - 1, 3, float("inf")), (L - 1, 77, float("nan")), (max(0, L - 2), 5, -float("inf"))):
            b.v[int(b.table[s, p // 16]), p % 16, 0, d] = bad
    out, lse2 = b.attention()
    assert_status_ok()
    assert torch.equal(lse, lse2)
    for t in range(b.T):
        ahead = b.lens[b.seq[t]] - 1 - b.pos[t]
        want = clean[t].clone()
        if ahead < 1:
            want[:, 3], want[:, 77] = float("inf"), float("nan")
        if ahead < 2:
            want[:, 5] = -float("inf")
        assert torch.equal(out[t].nan_to_num(nan=123.0), want.nan_to_num(nan=123.0)), t


def test_same_bits_again_on_another_stream_and_in_a_graph():
    b = Batch([3000, 1200, 5], _last([3000, 1200, 5], 2), 16, 2, 128, 16, BF)
    out, lse, ws = b.buffers()
    run = lambda: misa.attention(b.prob, b.cache, b.q, out, ws, lse=lse)
    run()
    torch.cuda.synchronize()
    want, wl = out.clone(), lse.clone()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        out.zero_()
        run()
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for _ in range(3):
        out.zero_()
        ws.fill_(0xff)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)
    # the captured call follows the device's positions
    b.prob.q_pos.sub_(1).clamp_(min=0)
    g.replay()
    torch.cuda.synchronize()
    b.pos = np.maximum(b.pos - 1, 0)
    b.check(out, lse)


def test_offsets_past_32_bits():
    # page_stride * page beyond 2^31 elements: 40 pages of 64 MiB-element stride (fp16, 5 GB of cache)
    stride = 1 << 26
    try:
        base = torch.zeros(40 * stride + 16 * 64, dtype=FP, device="cuda")
    except torch.OutOfMemoryError:
        pytest.skip("no room")
    view = lambda x: x.as_strided((40, 16, 1, 64), (stride, 64, 64, 1))
    k = view(base)
    v = view(base[2048:].as_strided((39 * stride + 1024,), (1,)))
    b = Batch([600], [[599]], 8, 1, 64, 16, FP, spare_pages=2)
    table = torch.arange(39, -1, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    for j in range(38):
        n = min(16, 600 - 16 * j)
        k[39 - j, :n] = b.tok_k[0][16 * j:16 * j + n].cuda()
        v[39 - j, :n] = b.tok_v[0][16 * j:16 * j + n].cuda()
    b.cache = misa.KVCache(k, v, table)
    out, lse = b.attention()
    assert_status_ok()
    b.check(out, lse)


def test_a_step_as_it_is_used():
    """Append to both caches, pool, route, select, attend; then the same step as one graph."""
    g = torch.Generator().manual_seed(3)
    lens, n = [900, 400], 2
    b = Batch(lens, _last(lens, n), 16, 2, 128, 16, BF)
    H, m, k = 16, 8, 128
    prob = misa.Problem(lens, [0, n, 2 * n], b.pos, num_heads=H, block=64)
    rand = lambda *s: torch.randn(s, generator=g).to(BF).cuda()
    K = rand(sum(lens), 1, 128)
    new_k, new_v, index_k, q, iq = rand(4, 2, 128), rand(4, 2, 128), rand(4, 1, 128), rand(4, 16, 128), rand(4, H, 128)
    w = torch.randn(4, H, generator=g).cuda()
    rope = misa.rope_table(1000, 128)
    index_cache = misa.KVCache(K)
    ix = misa.Indexer(prob, m=m, k=k)
    misa.pool_keys(prob, K, ix.Kbar)
    q_out, iq_out = torch.empty_like(q), torch.empty_like(iq)
    new_from = torch.tensor([L - n for L in lens], dtype=torch.int32, device="cuda")

    def step():
        misa.cache_append(prob, b.cache, new_k, new_v, q=q, q_out=q_out, rope=rope)
        misa.cache_append(prob, index_cache, index_k, q=iq, q_out=iq_out, rope=rope)
        ix.misa(iq_out, w, K, pool_from=new_from)
        return ix.attend(q_out, b.cache)

    out = step()
    assert_status_ok()
    want = out.clone()
    # the same, from the cache as it now is
    b.q_host = q_out.cpu()
    ko = [0, lens[0]]
    for t in range(4):
        s, p = b.seq[t], b.pos[t]
        at = int(b.table[s, p // 16]), p % 16
        b.tok_k[s][p], b.tok_v[s][p] = b.k[at].cpu(), b.v[at].cpu()
        assert torch.equal(b.v[at], new_v[t]) and not torch.equal(K[ko[s] + p], index_k[t])
    idx = ix.idx.cpu().numpy()
    assert all(len(set(r)) == k and r.max() <= b.pos[t] for t, r in enumerate(idx))
    lse = torch.empty(4, 16, device="cuda")
    ix.attend(q_out, b.cache, lse=lse)
    b.check(out, lse, idx=idx)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert_status_ok()
    # rows of idx come in no fixed order, so the sums may differ in their last bits
    assert torch.equal(torch.from_numpy(np.sort(idx, 1)), ix.idx.cpu().sort(1).values)
    b.check(out, lse, idx=ix.idx.cpu().numpy())
    assert (out.float() - want.float()).abs().max() <= 2.0 ** -6 * want.float().abs().max()


@pytest.mark.parametrize("hq", [4, 56])                # warp-level and tcgen05 kernels
@pytest.mark.parametrize("scale", [-0.07, 0.0, 0.3])
def test_scales_of_any_sign(hq, scale):
    b = Batch([700, 333], _last([700, 333], 2), hq, 1, 128, 16, BF)
    out, lse = b.attention(scale=scale)
    assert_status_ok()
    b.check(out, lse, scale=scale)
    idx = _lists(b, 150, 1)
    out, lse = b.selected(idx, scale=scale)
    b.check(out, lse, idx=idx, scale=scale)


@pytest.mark.parametrize("hq,n", [(4, 1), (8, 9)])
def test_more_sequences_than_a_warp(hq, n):
    g = np.random.default_rng(5)
    lens = [int(x) for x in g.integers(n, 400, 70)]
    b = Batch(lens, _last(lens, n), hq, 1, 64, 16, BF, seed=6, pad_rows=3)
    out, lse = b.attention()
    assert_status_ok()
    b.check(out, lse)
    # and as many groups: pairs of sequences that share, in turn with ones that do not
    prefix = {s: (s + 2, min(lens[s], lens[s + 1]) // 2) for s in range(0, 69, 3)}
    b = Batch(lens, _last(lens, n), hq, 1, 64, 16, BF, seed=6, pad_rows=3, prefix=prefix)
    so, ln = [0], []
    for s in range(0, 69, 3):
        so += [s + 2, s + 3]
        ln += [prefix[s][1], 0]
    share = misa.SharedPrefix(so, ln)
    out, lse = b.attention(share=share)
    assert_status_ok()
    b.check(out, lse)


def test_shared_lengths_that_do_not_hold_are_flagged_and_cut():
    for hq in (4, 64):
        b = Batch([100, 120], _last([100, 120], 1), hq, 1, 64, 16, BF, prefix={0: (2, 100)})
        share = misa.SharedPrefix([0, 2], [117], max_len=118)   # the first sequence has 100
        out, lse = b.attention(share=share)
        assert misa.stream_status()[1] == 0x4
        b.check(out, lse)
        share = misa.SharedPrefix([0, 2], [100], max_len=64)
        out, lse = b.attention(share=share)
        assert misa.stream_status()[1] == 0x4
        b.check(out, lse)


@pytest.mark.parametrize("hq", [4, 64])
@pytest.mark.parametrize("extra", [8, 64, 136])
def test_pages_with_gaps_between_them(hq, extra):
    """Page strides that are no multiple of a row's elements, or only of their half."""
    b = Batch([333, 90], _last([333, 90], 3), hq, 1, 128, 16, BF)
    count = b.k.shape[0]
    step = 16 * 128 + extra
    k, v = (torch.full((count * step,), float("nan"), dtype=BF, device="cuda").as_strided((count, 16, 1, 128), (step, 128, 128, 1))
            for _ in range(2))
    k.copy_(b.k)
    v.copy_(b.v)
    b.cache = misa.KVCache(k, v, b.table_dev)
    out, lse = b.attention()
    assert_status_ok()
    b.check(out, lse)
    idx = _lists(b, 60, 2)
    out, lse = b.selected(idx)
    b.check(out, lse, idx=idx)


def test_no_queries_and_no_tokens():
    b = Batch([50, 0], [[], []], 4, 2)
    out, lse = b.attention()
    idx = np.zeros((0, 5), np.int32)
    b.selected(idx)
    assert_status_ok() is None and out.numel() == 0


def test_two_streams_at_once():
    """Different calls in flight together, each with a workspace of its own."""
    batches = [Batch([20000, 500], _last([20000, 500], 2), 8, 1, 128, 64, BF, seed=1),
               Batch([900, 1200], _last([900, 1200], 60), 8, 1, 128, 16, FP, seed=2),
               Batch([3000], _last([3000], 3), 64, 1, 64, 16, BF, seed=3)]
    idx = torch.from_numpy(_lists(batches[2], 700, 4)).cuda()
    bufs = [b.buffers() for b in batches[:2]] + [batches[2].buffers(700)]

    def run(i):
        b, (out, lse, ws) = batches[i], bufs[i]
        if i == 2:
            misa.attention_selected(b.prob, b.cache, b.q, idx, out, ws, lse=lse)
        else:
            misa.attention(b.prob, b.cache, b.q, out, ws, lse=lse)

    for i in range(3):
        run(i)
    torch.cuda.synchronize()
    want = [(o.clone(), l.clone()) for o, l, _ in bufs]
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        for o, l, _ in bufs:
            o.zero_()
        torch.cuda.synchronize()
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                run(i)
        torch.cuda.synchronize()
        for (o, l, _), (wo, wl) in zip(bufs, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)
    assert_status_ok()
    batches[0].check(*bufs[0][:2])
    batches[1].check(*bufs[1][:2])
    batches[2].check(*bufs[2][:2], idx=idx.cpu().numpy())


def test_one_workspace_in_two_graphs_of_one_stream():
    b = Batch([9000, 4000], _last([9000, 4000], 2), 8, 1, 128, 64, BF)
    c = Batch([700, 900], _last([700, 900], 70), 8, 1, 128, 64, BF, seed=9)
    (o1, l1, w1), (o2, l2, w2) = b.buffers(), c.buffers()
    ws = w1 if w1.numel() >= w2.numel() else w2
    runs = [lambda: misa.attention(b.prob, b.cache, b.q, o1, ws, lse=l1),
            lambda: misa.attention(c.prob, c.cache, c.q, o2, ws, lse=l2)]
    graphs = []
    for r in runs:
        r()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r()
        graphs.append(g)
    for _ in range(3):
        o1.zero_()
        o2.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        b.check(o1, l1)
        c.check(o2, l2)
    assert_status_ok()


@pytest.mark.parametrize("hq", [4, 64])
def test_queries_inside_the_shared_prefix(hq):
    lens, qs = [300, 280, 400], [[10, 299], [5, 130, 255], [256, 0]]
    b = Batch(lens, qs, hq, 1, 128, 16, BF, prefix={0: (3, 256)})
    share = misa.SharedPrefix([0, 3], [256])
    opts = dict(softcap=20.0, slopes=_slopes(hq))
    for kw in ({}, opts):
        out, lse = b.attention(share=share, **kw)
        assert_status_ok()
        b.check(out, lse, **kw)


def test_calls_that_python_or_the_library_refuse():
    b = Batch([50, 40], _last([50, 40], 1), 4, 2)
    with pytest.raises(ValueError, match="page_table"):
        misa.KVCache(b.k, b.v, b.table_dev[:1].expand(2, -1))
    out, lse, ws = b.buffers()
    with pytest.raises(misa.MisaError, match="out must not be q"):
        misa.attention(b.prob, b.cache, b.q, b.q, ws)
    with pytest.raises(misa.MisaError, match="workspace too small"):
        big = Batch([30000], [[29999]], 4, 1)
        misa.attention(big.prob, big.cache, big.q, big.buffers()[0], ws)
    b.attention()
    assert_status_ok()
