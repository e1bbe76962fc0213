"""Ragged batches for the cache and attention tests, and their error bounds."""
import numpy as np
import torch

import long_context_sparse_misa_b200 as misa
from oracle import attention as plain

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


class Batch:
    """Sequences of the given lengths; queries[s] positions of sequence s.
    Pages are in random order and the cache beyond every sequence holds NaN."""

    def __init__(self, lens, queries, hq, hkv, dim=128, page=16, dtype=torch.bfloat16, seed=0,
                 heads_first=False, spare_pages=3, pad_rows=0, packed=False, prefix=None,
                 fill=float("nan")):
        g = np.random.default_rng(seed)
        self.lens, self.queries, self.hq, self.hkv, self.dim = lens, queries, hq, hkv, dim
        self.dtype, self.page = dtype, page
        S = len(lens)
        self.seq = np.concatenate([[s] * len(q) for s, q in enumerate(queries)] + [[]]).astype(int)
        self.pos = np.concatenate([np.asarray(q, np.int64) for q in queries] + [np.zeros(0, np.int64)]).astype(int)
        self.T = len(self.pos)
        offsets = np.concatenate([[0], np.cumsum([len(q) for q in queries])])
        pos = np.concatenate([self.pos, np.full(pad_rows, 7)])
        self.prob = misa.Problem(lens, offsets, pos, num_heads=1, block=64)
        self.rows = self.T + pad_rows

        def values(*shape):
            return torch.from_numpy(g.standard_normal(shape, dtype=np.float32)).to(dtype)

        self.tok_k = [values(n, hkv, dim) for n in lens]
        self.tok_v = [values(n, hkv, dim) for n in lens]
        if prefix:  # {first sequence: (one past the last, length)}: the same tokens
            for a, (b, n) in prefix.items():
                for s in range(a + 1, b):
                    self.tok_k[s][:n], self.tok_v[s][:n] = self.tok_k[a][:n], self.tok_v[a][:n]
        if packed:
            flat = lambda xs: torch.cat(xs + [values(0, hkv, dim)]).cuda()
            self.table = None
            self.k, self.v = flat(self.tok_k), flat(self.tok_v)
            self.cache = misa.KVCache(self.k, self.v)
        else:
            need = [-(-n // page) for n in lens]
            wide = max(1, max(need))
            order = g.permutation(sum(need) + spare_pages)
            self.table = np.full((S, wide), -1, np.int32)
            at = 0
            for s, n in enumerate(need):
                self.table[s, :n] = order[at:at + n]
                at += n
            count = sum(need) + spare_pages
            shape = (count, hkv, page, dim) if heads_first else (count, page, hkv, dim)

            def pool(toks):
                c = torch.full(shape, fill, dtype=dtype)
                view = c.transpose(1, 2) if heads_first else c
                for s, n in enumerate(lens):
                    for j in range(need[s]):
                        part = toks[s][j * page:(j + 1) * page]
                        view[int(self.table[s, j]), :len(part)] = part
                c = c.cuda()
                return c.transpose(1, 2) if heads_first else c

            self.k, self.v = pool(self.tok_k), pool(self.tok_v)
            self.table_dev = torch.from_numpy(self.table).cuda()
            self.cache = misa.KVCache(self.k, self.v, self.table_dev)
        self.q_host = values(self.rows, hq, dim)
        self.q = self.q_host.cuda()

    def buffers(self, k=0, share=None):
        out = torch.full((self.rows, self.hq, self.dim), 7.0, dtype=self.dtype, device="cuda")
        lse = torch.full((self.rows, self.hq), 7.0, device="cuda")
        ws = torch.full((misa.attention_workspace_size(self.prob, self.cache, self.hq, k, share),), 0xff,
                        dtype=torch.uint8, device="cuda")
        return out, lse, ws

    def attention(self, share=None, **kw):
        out, lse, ws = self.buffers(0, share)
        misa.attention(self.prob, self.cache, self.q, out, ws, lse=lse, share=share, **kw)
        return out, lse

    def selected(self, idx, **kw):
        out, lse, ws = self.buffers(idx.shape[1])
        misa.attention_selected(self.prob, self.cache, self.q, torch.from_numpy(idx).cuda(), out, ws,
                                lse=lse, **kw)
        return out, lse

    def check(self, out, lse, idx=None, scale=None, softcap=0.0, slopes=None, rows=None):
        """Against the definition in 64 bits, every element of every row.

        With u the type's half step: each weight is rounded once (u sum p |v|)
        and the result once (u |out|).  An exponent is off by d = dim 2^-22
        sum |q k| scale (an fp32 sum of dim products, each addition off by at
        most 2^-23 of what is summed, and as much again for the scaling) plus
        2^-20 (max |x| + cap + 1) for the cap, the bias, the exponential and
        the joining; weights are then off by e^{2d} - 1 <= 2.1 d relative."""
        o, l = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        scale = self.dim ** -0.5 if scale is None else scale
        s_host = None if slopes is None else slopes.cpu().numpy().astype(np.float64)
        u = HALF_STEP[self.dtype]
        f = lambda x: x.float().numpy()
        for t in (range(self.T) if rows is None else rows):
            s, pos = self.seq[t], self.pos[t]
            tok = np.arange(pos + 1) if idx is None else idx[t][(idx[t] >= 0) & (idx[t] <= pos)]
            want, wl, spread, reach, top = plain.attend(
                f(self.q_host[t]), f(self.tok_k[s])[tok], f(self.tok_v[s])[tok], pos, tok, scale, softcap, s_host)
            d = self.dim * 2.0 ** -22 * reach + 2.0 ** -20 * (top + softcap + 1)
            tol = (u + 2.1 * d[:, None]) * spread + u * np.abs(want) * (1 + u) + 1e-30
            if self.dtype == torch.float16:  # below 2^-14 half a step is 2^-25, of a weight and of the result
                tol = tol + 2.0 ** -25 * (1 + np.abs(f(self.tok_v[s])[tok]).sum(0).max() if len(tok) else 1)
            assert np.isfinite(o[t]).all(), f"row {t}: not finite"
            err = np.abs(o[t] - want)
            assert (err <= tol).all(), f"row {t} (sequence {s}, position {pos}): {(err / tol).max():.2f} x its bound"
            if len(tok):
                assert (np.abs(l[t] - wl) <= 2.1 * d + 2.0 ** -20 * np.abs(wl)).all(), f"row {t}: lse"
            else:
                assert (o[t] == 0).all() and (l[t] == -np.inf).all(), f"row {t}: sees nothing"
        for t in range(self.T, self.rows):
            assert (o[t] == 7).all() and (l[t] == 7).all(), f"padding row {t} was written"


def status():
    return misa.stream_status()


def assert_status_ok():
    code, bits = misa.stream_status()
    assert code == 0 and bits == 0, f"device status {code}/{bits}"
