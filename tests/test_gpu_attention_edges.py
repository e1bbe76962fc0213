"""The cache and attention entry points on a B200 in corners of what their
documentation allows: empty tables, padding rows that are not there, values
that are not finite, caps and weights at the ends of their range."""
import numpy as np
import pytest
import torch

import long_context_sparse_misa_b200 as misa
from tests.attention_cases import Batch, assert_status_ok

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
BOUNDS, BAD_INPUT = 0x2, 0x4


def _last(lens, n):
    return [list(range(max(0, L - n), L)) for L in lens]


def _slopes(hq):
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / hq) for i in range(hq)], device="cuda")


def _bits(x):
    return x.contiguous().view(torch.int16)


@pytest.mark.parametrize("hq", [4, 64])                # warp-level and tcgen05 kernels
def test_a_page_table_without_entries_has_room_for_no_token(hq):
    b = Batch([40, 23], _last([40, 23], 2), hq, 1, page=16)
    cache = misa.KVCache(b.k, b.v, b.table_dev[:, :0])
    before = b.k.clone(), b.v.clone()
    new = torch.ones(b.T, 1, 128, dtype=BF, device="cuda")
    misa.cache_append(b.prob, cache, new, new)
    assert misa.stream_status()[1] == BOUNDS
    assert torch.equal(_bits(b.k), _bits(before[0])) and torch.equal(_bits(b.v), _bits(before[1]))
    b.cache = cache
    out, lse = b.attention()
    assert misa.stream_status()[1] == BOUNDS
    assert (out == 0).all() and (lse == -float("inf")).all()
    out, lse = b.selected(np.tile(np.arange(5, dtype=np.int32), (b.T, 1)))
    assert misa.stream_status()[1] == BOUNDS
    assert (out == 0).all() and (lse == -float("inf")).all()


@pytest.mark.parametrize("live,pad", [(1, 2500), (700, 1300), (1200, 1), (0, 900)])
def test_append_with_blocks_of_padding_rows(live, pad):
    """Blocks that hold some padding rows, or nothing else; what those rows hold goes nowhere."""
    b = Batch([live + 5, 9], [list(range(live)), []], 2, 1, dim=64, page=16, pad_rows=pad)
    x = torch.randn(b.rows, 4, 64, device="cuda").to(BF)
    x[live:] = float("nan")
    q_out = torch.full((b.rows, 2, 64), 9.0, dtype=BF, device="cuda")
    want_k, want_v = b.k.clone(), b.v.clone()
    at = torch.arange(live, device="cuda")
    page = b.table_dev[0, at // 16].long()
    want_k[page, at % 16], want_v[page, at % 16] = x[:live, 2:3], x[:live, 3:4]
    misa.cache_append(b.prob, b.cache, x[:, 2:3], x[:, 3:4], q=x[:, :2], q_out=q_out)
    assert_status_ok()
    assert torch.equal(_bits(b.k), _bits(want_k)) and torch.equal(_bits(b.v), _bits(want_v))
    assert torch.equal(q_out[:live], x[:live, :2]) and (q_out[live:] == 9).all()


@pytest.mark.parametrize("k", [100, 200, 300])          # one, two and three tiles: even and odd shares of the two streams
@pytest.mark.parametrize("dim", [64, 128])
def test_blocks_that_take_many_lists_in_turn(k, dim):
    """More tcgen05 items than blocks, with queries that see nothing between them."""
    b = Batch([350, 200], [[300 + t % 50 for t in range(700)], [199] * 5], 48, 1, dim, 16, BF)
    g = np.random.default_rng(k)
    idx = np.stack([g.permutation(301)[:k] if t < 700 else g.permutation(400)[:k] % 200 for t in range(b.T)]).astype(np.int32)
    blind = np.arange(3, 700, 7)
    idx[blind[::2]] = -1
    b.prob.q_pos[torch.from_numpy(blind[1::2].copy()).cuda()] = -1
    out, lse = b.selected(idx)
    assert misa.stream_status()[1] == BAD_INPUT
    assert (out[blind] == 0).all() and (lse[blind] == -float("inf")).all()
    b.check(out, lse, idx=idx, rows=[t for t in range(0, b.T, 23) if t not in blind] + list(range(700, 705)))
    for t in range(2, 9):                               # other rows: the same list alone gives the same bits
        one = np.full_like(idx, -1)
        one[t * 50] = idx[t * 50]
        if t * 50 not in blind:
            alone, l1 = b.selected(one)
            assert torch.equal(alone[t * 50], out[t * 50]) and torch.equal(l1[t * 50], lse[t * 50])
    misa.stream_status()


# ---------------------------------------------------------------- what is not finite, under a cap
ROWS = [(4, 1), (16, 1), (8, 3), (32, 2), (8, 20), (48, 1)]  # query heads on one key head, queries: 4 to 160 rows


@pytest.mark.parametrize("hq,n", ROWS)
@pytest.mark.parametrize("dt", [BF, FP])
def test_a_nan_in_one_row_of_q_stays_there_under_a_cap(hq, n, dt):
    b = Batch([400, 333], _last([400, 333], n), hq, 1, page=16, dtype=dt)
    opts = dict(softcap=20.0, slopes=_slopes(hq))
    idx = np.stack([np.arange(150, dtype=np.int32)] * b.T)
    for run in (lambda: b.attention(**opts), lambda: b.selected(idx, **opts)):
        clean, lse = run()
        assert_status_ok()
        for t, h in ((0, 0), (b.T - 1, hq // 2), (n // 2, hq - 1)):
            kept = b.q[t, h].clone()
            b.q[t, h, 5] = float("nan")
            out, lse2 = run()
            b.q[t, h] = kept
            assert out[t, h].isnan().all() and lse2[t, h].isnan()
            out[t, h], lse2[t, h] = clean[t, h], lse[t, h]
            assert torch.equal(out, clean) and torch.equal(lse2, lse), (t, h)
    assert_status_ok()


@pytest.mark.parametrize("seqs,hq", [(4, 4), (12, 2), (3, 16), (40, 4)])
def test_a_nan_in_one_sequence_stays_there_under_a_cap_with_a_shared_prefix(seqs, hq):
    lens = [260 + 7 * (s % 5) for s in range(seqs)]
    b = Batch(lens, _last(lens, 1), hq, 1, page=16, prefix={0: (seqs, 256)})
    share = misa.SharedPrefix([0, seqs], [256])
    clean, lse = b.attention(share=share, softcap=30.0)
    assert_status_ok()
    for t in (0, seqs // 2, seqs - 1):
        kept = b.q[t].clone()
        b.q[t, 0, 100] = float("nan")
        out, lse2 = b.attention(share=share, softcap=30.0)
        b.q[t] = kept
        assert out[t, 0].isnan().all() and lse2[t, 0].isnan()
        out[t, 0], lse2[t, 0] = clean[t, 0], lse[t, 0]
        assert torch.equal(out, clean) and torch.equal(lse2, lse), t


@pytest.mark.parametrize("hq,n", ROWS)
def test_an_infinite_key_is_a_capped_score(hq, n):
    """Infinities give the cap or minus the cap, as any product far beyond it does; only a row whose
    query has a zero there gets a NaN.  Rows of a tile that do not exist hold zeros."""
    b = Batch([400, 333], _last([400, 333], n), hq, 1, page=16)
    b.q[b.T - 1, hq - 1, 9] = 0
    at = int(b.table[0, 2]), 5
    idx = np.stack([np.arange(150, dtype=np.int32)] * b.T)
    for run in (lambda: b.attention(softcap=15.0), lambda: b.selected(idx, softcap=15.0)):
        for sign in (1.0, -1.0):
            for s in range(2):
                at = int(b.table[s, 2]), 5
                b.k[at][0, 9] = sign * 2.0 ** 60
            want, wl = run()
            for s in range(2):
                at = int(b.table[s, 2]), 5
                b.k[at][0, 9] = sign * float("inf")
            out, lse = run()
            assert out[b.T - 1, hq - 1].isnan().all()
            out[b.T - 1, hq - 1], lse[b.T - 1, hq - 1] = want[b.T - 1, hq - 1], wl[b.T - 1, hq - 1]
            assert torch.equal(out, want) and torch.equal(lse, wl)
    assert_status_ok()


@pytest.mark.parametrize("hq,n", [(2, 3), (8, 2), (16, 3), (16, 2), (4, 150)])
def test_what_the_last_token_holds_reaches_no_earlier_query_under_a_cap(hq, n):
    b = Batch([400, 333], _last([400, 333], n), hq, 1, page=16)
    clean, lse = b.attention(softcap=20.0)
    for s, L in enumerate(b.lens):
        at = int(b.table[s, (L - 1) // 16]), (L - 1) % 16
        b.k[at], b.v[at] = float("nan"), float("inf")
    out, lse2 = b.attention(softcap=20.0)
    assert_status_ok()
    early = [t for t in range(b.T) if b.pos[t] < b.lens[b.seq[t]] - 1]
    assert torch.equal(out[early], clean[early]) and torch.equal(lse[early], lse2[early])
    late = [t for t in range(b.T) if b.pos[t] == b.lens[b.seq[t]] - 1]
    assert out[late].isnan().all()


# ---------------------------------------------------------------- caps of any size
def _check_cap(b, out, lse, idx=None, rows=None, softcap=0.0, scale=None, slopes=None):
    """Batch.check with a bound that does not grow with the cap.

    Half steps as there.  An exponent is off by dim 2^-22 sum |q k| scale for its product (the cap
    makes no error larger), 2^-20 (max |x| + 1) for the bias, the exponential and the joining, and for
    the cap itself by a share of |x|: its series by 8 roundings (2^-21); its quotient 2 cap / (e + 1),
    at most 2 cap, by 8 roundings and the exponential's 2^-22, so 2^-20 cap in all, where |x| is at least
    cap tanh(1/2) = 0.46 cap: 3 2^-20 |x|.  Together under 2^-18 (max |x| + 1)."""
    from oracle import attention as plain
    from tests.attention_cases import HALF_STEP
    u = HALF_STEP[b.dtype]
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    f = lambda x: x.float().numpy()
    scale = b.dim ** -0.5 if scale is None else scale
    s_host = None if slopes is None else slopes.double().cpu().numpy()
    for t in range(b.T) if rows is None else rows:
        s, pos = b.seq[t], b.pos[t]
        tok = np.arange(pos + 1) if idx is None else idx[t][(idx[t] >= 0) & (idx[t] <= pos)]
        want, wl, spread, reach, top = plain.attend(f(b.q_host[t]), f(b.tok_k[s])[tok], f(b.tok_v[s])[tok], pos, tok,
                                                    scale, softcap, s_host)
        d = b.dim * 2.0 ** -22 * reach + 2.0 ** -18 * (top + 1)
        assert (d < 0.1).all()                           # the bound below is of first order
        tol = (u + 2.2 * d[:, None]) * spread + u * np.abs(want) * (1 + u) + 1e-30
        if b.dtype == FP:
            tol = tol + 2.0 ** -25 * (1 + np.abs(f(b.tok_v[s])[tok]).sum(0).max())
        err = np.abs(o[t] - want)
        assert (err <= tol).all(), f"row {t}: {(err / tol).max():.2f} x its bound"
        assert (np.abs(l[t] - wl) <= 2.2 * d + 2.0 ** -20 * np.abs(wl)).all(), f"row {t}: lse"


CAPS = [(65.0, None), (65.0, 1.5), (200.0, 3.0), (200.0, -3.0), (1e3, None), (1e3, 3.0), (1e4, None), (1e6, None), (1e8, None),
        (3e38, None), (1e-3, None), (1e-30, None), (1e-40, None)]


@pytest.mark.parametrize("softcap,scale", CAPS)
@pytest.mark.parametrize("hq,n,dt", [(4, 2, FP), (16, 1, BF), (48, 1, FP), (4, 40, BF)])
def test_caps_of_any_size(softcap, scale, hq, n, dt):
    b = Batch([300, 131], _last([300, 131], n), hq, 1, 64, 16, dt, seed=3)
    b.q_host[0, 1] = 0                                   # products of 0 stay 0, whatever the cap
    b.q = b.q_host.cuda()
    rows = sorted({0, 1, b.T // 2, b.T - 1})
    opts = dict(softcap=softcap, scale=scale, slopes=_slopes(hq))
    out, lse = b.attention(**opts)
    assert_status_ok()
    _check_cap(b, out, lse, rows=rows, **opts)
    idx = np.stack([np.arange(120, dtype=np.int32)] * b.T)
    out, lse = b.selected(idx, softcap=softcap, scale=scale)
    assert misa.stream_status()[1] == (BAD_INPUT if (b.pos < 119).any() else 0)  # some lists name tokens ahead
    _check_cap(b, out, lse, idx=idx, rows=rows, softcap=softcap, scale=scale)


# ---------------------------------------------------------------- many small weights behind a large one
@pytest.mark.parametrize("nats", [16.23, 17.0, 18.5])
@pytest.mark.parametrize("heads,grp,seqs,sink", [(8, 1, 64, 0), (4, 48, 40, -1), (4, 48, 40, 0)])
@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("dt", [BF, FP])
def test_many_small_weights_behind_a_large_one(nats, heads, grp, seqs, sink, listed, dt):
    """One token with a value of zero takes nearly all the weight, the others' small ones make the result.

    N equal weights w = e^-x of the others, values c[d]: out = c N w / (1 + N w).  Each weight is rounded to
    the type by half a step u of itself, or by half of fp16's smallest step, 2^-25: 2^-40 of the largest weight in
    the warp-level kernel (weights up to 2^15), 2^-32 in the tcgen05 one (its reference times 2^7).  Its exponent
    is off by d = 2^-22 dim x + 2^-20 (x + 1), fp32 sums of N / 16 terms at most by 2^-24 N / 16, the result by
    half a step of its own."""
    n = 65536 if listed else 100000
    dim, page, hq = 64, 64, heads * grp
    u = {BF: 2.0 ** -8, FP: 2.0 ** -11}[dt]
    pages = -(-n // page)
    k = torch.zeros(pages, page, heads, dim, dtype=dt, device="cuda")
    c = (0.5 + torch.arange(dim) / 64).to(dt)
    v = c.cuda().expand(pages, page, heads, dim).contiguous()
    place = sink % n
    k[place // page, place % page, :, 0] = nats
    v[place // page, place % page] = 0
    q = torch.zeros(seqs, hq, dim, dtype=dt, device="cuda")
    q[:, :, 0] = 8.0
    x = 8.0 * float(k[place // page, place % page, 0, 0]) / 8.0   # scale 1/8
    prob = misa.Problem([n] * seqs, range(seqs + 1), [n - 1] * seqs, num_heads=1, block=64)
    cache = misa.KVCache(k, v, torch.arange(pages, dtype=torch.int32, device="cuda").repeat(seqs, 1))
    out, lse = torch.empty_like(q), torch.empty(seqs, hq, device="cuda")
    ws = torch.empty(misa.attention_workspace_size(prob, cache, hq, n if listed else 0), dtype=torch.uint8, device="cuda")
    if listed:
        idx = torch.arange(n, dtype=torch.int32, device="cuda").repeat(seqs, 1)
        misa.attention_selected(prob, cache, q, idx, out, ws, lse=lse)
    else:
        misa.attention(prob, cache, q, out, ws, lse=lse)
    assert_status_ok()
    many = (n - 1) * np.exp(-x)
    want = c.double().numpy() * many / (1 + many)
    d = 2.0 ** -22 * dim * x + 2.0 ** -20 * (x + 1)
    small = 0.0 if dt == BF else 2.0 ** -32 if grp >= 48 else 2.0 ** -40
    tol = (u + 2.1 * d + 2.0 ** -24 * n / 16 + small * np.exp(x)) * want + u * want * (1 + u) + 2.0 ** -25
    err = np.abs(out.double().cpu().numpy() - want)
    assert (err <= tol).all(), f"{(err / tol).max():.2f} x its bound, off by {(err / want).max():.4f} of the value"
    assert (lse.double() - (x + np.log1p(many))).abs().max() <= 2.1 * d + 2.0 ** -20 * (x + 1)


# ---------------------------------------------------------------- groups and streams
def test_a_group_without_sequences_has_no_length_to_check():
    b = Batch([100, 120], _last([100, 120], 1), 4, 1, 64, 16, BF, prefix={0: (2, 96)})
    for so, ln in (([0, 2, 2], [96, 50]), ([0, 0, 2], [110, 96]), ([0, 0, 2, 2, 2], [120, 96, 5, 7])):
        out, lse = b.attention(share=misa.SharedPrefix(so, ln))
        assert_status_ok()
        b.check(out, lse)


def test_attend_on_a_stream_of_its_own_takes_no_memory_that_is_still_written():
    """The buffers that Indexer.attend makes at its first call belong to the stream it runs on: memory that
    the current stream has freed, but not yet written for the last time, is not among them."""
    b = Batch([900, 400], _last([900, 400], 2), 16, 2, 128, 16, BF)
    prob = misa.Problem(b.lens, [0, 2, 4], b.pos, num_heads=8, block=64)
    ix = misa.Indexer(prob, m=8, k=128)
    ix.idx.copy_(torch.from_numpy(np.stack([np.arange(128, dtype=np.int32)] * 4)))
    want, _ = b.selected(ix.idx.cpu().numpy())
    q = b.q.repeat(1, 1, 1)
    size = misa.attention_workspace_size(prob, b.cache, 16, 128)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)                       # about 0.2 s
    stale = [torch.empty(size, dtype=torch.uint8, device="cuda"), torch.empty_like(q)]
    for x in stale:
        x.fill_(0x7f)
    del stale, x
    out = ix.attend(q, b.cache, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_no_queries_give_no_rows():
    b = Batch([50, 0], [[], []], 4, 2)
    out, lse = b.attention(softcap=3.0)
    assert out.shape == (0, 4, 128) and lse.shape == (0, 4)
    out, lse = b.selected(np.zeros((0, 5), np.int32))
    assert out.shape == (0, 4, 128) and lse.shape == (0, 4)
    assert_status_ok()


@pytest.mark.parametrize("hq", [4, 64])                # warp-level and tcgen05 kernels
@pytest.mark.parametrize("dt,softcap", [(FP, 0.0), (BF, 90.0)])
def test_sequences_that_end_inside_their_groups_prefix(hq, dt, softcap):
    """They share what they have of it."""
    lens, qs = [300, 100, 257, 17], [[299], [99, 3], [256, 255], [16]]
    b = Batch(lens, qs, hq, 1, 64, 16, dt, pad_rows=2)
    for s in range(1, 4):                               # read where the first sequence keeps them
        n = min(lens[s], 256)
        b.tok_k[s][:n], b.tok_v[s][:n] = b.tok_k[0][:n], b.tok_v[0][:n]
    out, lse = b.attention(share=misa.SharedPrefix([0, 4], [256]), softcap=softcap)
    assert_status_ok()
    b.check(out, lse, softcap=softcap)


@pytest.mark.parametrize("hq", [4, 64])
@pytest.mark.parametrize("softcap", [0.0, 25.0, 5000.0])
def test_a_padded_batch_in_a_graph_with_other_values(hq, softcap):
    """Captured once, replayed on other queries; padding rows hold NaN and are left alone."""
    b = Batch([700, 90], _last([700, 90], 2), hq, 1, 128, 16, FP, pad_rows=5)
    b.q[b.T:] = float("nan")
    out, lse, ws = b.buffers()
    run = lambda o, l: misa.attention(b.prob, b.cache, b.q, o, ws, lse=l, softcap=softcap)
    run(out, lse)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run(out, lse)
    for seed in range(3):
        b.q[:b.T] = torch.randn(b.T, hq, 128, generator=torch.Generator().manual_seed(seed)).to(FP).cuda()
        want, wl, _ = b.buffers()
        run(want, wl)
        out.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)
        assert (out[b.T:] == 7).all() and (lse[b.T:] == 7).all() and out[:b.T].isfinite().all()
    assert_status_ok()


def test_wide_caps_come_close_to_none():
    b = Batch([500, 200], _last([500, 200], 3), 16, 1, 128, 16, FP)
    none, lse = b.attention()
    wide, lse2 = b.attention(softcap=1e30)
    assert_status_ok()
    # the same exponents but for a rounding of each of their factors, some 2^-22 of at most 8
    assert (lse - lse2).abs().max() <= 2.0 ** -17
    assert (none.float() - wide.float()).abs().max() <= 2.0 ** -10 * none.float().abs().max()


@pytest.mark.parametrize("hq", [4, 64])
def test_one_head_in_either_order_of_tokens_and_heads(hq):
    b = Batch([300, 77], _last([300, 77], 2), hq, 1, 64, 16, BF)
    want, lse = b.attention()
    b.cache = misa.KVCache(b.k, b.v.transpose(1, 2).contiguous().transpose(1, 2), b.table_dev)
    out, lse2 = b.attention()
    assert_status_ok()
    assert torch.equal(out, want) and torch.equal(lse, lse2)


@pytest.mark.parametrize("hq", [4, 48])                # warp-level and tcgen05 kernels
def test_lse_of_equal_scores_in_fp16(hq):
    """Scores of 0: lse is the logarithm of the number of tokens.  Held near log2 of it, 9 to 15.7, where a step is 2^-20:
    half one for lg2, joining and conversion each, and lg2's own error of as much: under 2^-20 on average over many
    numbers; 15 above that, where a step is twice as large, every other one was off by more."""
    lens = [int(n) for n in np.random.default_rng(2).integers(600, 50000, 64)]
    n = max(lens)
    pages = -(-n // 64)
    k = torch.zeros(pages, 64, 1, 64, dtype=FP, device="cuda")
    prob = misa.Problem(lens, range(65), [x - 1 for x in lens], num_heads=1, block=64)
    cache = misa.KVCache(k, torch.ones_like(k), torch.arange(pages, dtype=torch.int32, device="cuda").repeat(64, 1))
    q = torch.zeros(64, hq, 64, dtype=FP, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(64, hq, device="cuda")
    ws = torch.empty(misa.attention_workspace_size(prob, cache, hq), dtype=torch.uint8, device="cuda")
    misa.attention(prob, cache, q, out, ws, lse=lse)
    assert_status_ok()
    assert (out == 1).all()
    err = (lse.double().cpu() - torch.tensor(lens).double().log()[:, None]).abs()
    assert err.max() <= 3 * 2.0 ** -20 and err.mean() <= 2.0 ** -21, (float(err.mean()), float(err.max()))


@pytest.mark.parametrize("softcap", [15.0, 20.0, 30.0, 50.0, 64.0, 300.0])
@pytest.mark.parametrize("hq", [4, 48])                # warp-level and tcgen05 kernels
@pytest.mark.parametrize("dt", [BF, FP])
def test_a_capped_score_is_off_by_a_share_of_itself(softcap, hq, dt):
    """One token a sequence, so that lse is its score; the products are exact.

    Below half the cap eight roundings of the score (2^-21) and lse's conversion of two (2^-23); beyond, the
    quotient's share of 2^-20 of the cap, at most twice 2^-20 of the score / tanh(1/2) = 0.46.  fp16's weight, 2^15, is
    off by half a step of 15 (2^-21) and the exponential's 2^-22, its logarithm by as much again: under 2^-19."""
    S = 200
    b = Batch([1] * S, [[0]] * S, hq, 1, 64, 16, dt)
    b.q.zero_()
    b.q[:, :, 0] = 8.0                                   # times the scale of 1/8: the score is the key's first element
    g = torch.Generator().manual_seed(1)
    x = torch.cat([torch.randn(S // 2, generator=g) * 3, (torch.rand(S // 2, generator=g) - 0.5) * 3 * softcap]).to(dt)
    for s in range(S):
        b.k[int(b.table[s, 0]), 0, 0] = 0
        b.k[int(b.table[s, 0]), 0, 0, 0] = x[s]
    want = softcap * np.tanh(x.double().numpy() / softcap)
    tol = 2.0 ** -20 * np.abs(want) * np.where(np.abs(x.double().numpy()) < softcap / 2, 1, 2 / 0.46) + (2.0 ** -19 if dt == FP else 0)
    for out, lse in (b.attention(softcap=softcap), b.selected(np.zeros((S, 1), np.int32), softcap=softcap)):
        assert_status_ok()
        err = np.abs(lse.double().cpu().numpy() - want[:, None])
        assert (err <= tol[:, None]).all(), f"{(err / tol[:, None]).max():.2f} x its bound"
