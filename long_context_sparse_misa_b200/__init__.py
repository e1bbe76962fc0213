"""Python binding of libmisa, the B200 (sm_100a) MISA routed sparse-attention indexer.

Argument marshalling only: every step of the indexer runs in the CUDA
kernels behind the C ABI declared in include/misa.h.  PyTorch provides
device memory and streams.  There is no CPU fallback: importing this package
without a built libmisa.so raises ImportError (build it with
``python long_context_sparse_misa_b200/build.py``).

Method: "MISA: Mixture of Indexer Sparse Attention for Long-Context LLM
Inference" -- a block-pooled router keeps m of the H indexer heads per query,
only those heads score the causal prefix, and a per-query top-k follows;
MISA-dagger re-ranks an enlarged candidate set with all H heads; block
pruning lets the routed heads score only the tokens of the best pooled
blocks.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "LIB_PATH", "lib", "MisaError", "Problem", "workspace_size", "block_offsets", "pool_keys",
    "route", "pool_keys_from", "score_topk", "hier_rerank", "dsa_index_dense", "stream_status",
    "selftest_timeout", "route_static", "EXPORTED", "Indexer", "profile_enable", "profile_collect",
    "block_workspace_size", "block_score_topk",
    "KVCache", "SharedPrefix", "rope_table", "cache_append", "attention", "attention_selected",
    "attention_workspace_size",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmisa.so")

# Every symbol include/misa.h declares.
EXPORTED = (
    "misa_workspace_size", "misa_block_offsets", "misa_pool_keys", "misa_pool_keys_from",
    "misa_route",
    "misa_route_static", "misa_score_topk", "misa_hier_rerank", "dsa_index_dense", "misa_stream_status",
    "misa_selftest_timeout", "misa_profile_enable", "misa_profile_collect",
    "misa_last_error_string", "misa_block_workspace_size", "misa_block_score_topk",
    "misa_cache_append", "misa_attention", "misa_attention_selected",
    "misa_attention_workspace_size",
)

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with "
                      "`python long_context_sparse_misa_b200/build.py` (needs nvcc)")
lib = ctypes.CDLL(LIB_PATH)

_c_i32, _c_i64, _c_sz, _c_p = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p


class _Problem(ctypes.Structure):
    _fields_ = [
        ("num_seqs", _c_i32), ("num_queries", _c_i32), ("num_heads", _c_i32),
        ("head_dim", _c_i32), ("block", _c_i32), ("max_seq_len", _c_i32),
        ("total_keys", _c_i64), ("total_blocks", _c_i64),
        ("key_offsets", _c_p), ("block_offsets", _c_p), ("query_offsets", _c_p),
        ("q_pos", _c_p),
    ]


class _KVCache(ctypes.Structure):
    _fields_ = [
        ("k", _c_p), ("v", _c_p), ("dtype", _c_i32), ("num_kv_heads", _c_i32),
        ("head_dim", _c_i32), ("page_size", _c_i32), ("num_pages", _c_i32),
        ("pages_per_seq", _c_i32), ("page_table", _c_p), ("page_table_stride", _c_i64),
        ("page_stride", _c_i64), ("token_stride", _c_i64), ("head_stride", _c_i64),
    ]


class _AttentionOpts(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("slopes", _c_p)]


class _SharedPrefix(ctypes.Structure):
    _fields_ = [("num_groups", _c_i32), ("max_len", _c_i32), ("seq_offsets", _c_p),
                ("lens", _c_p)]


_PP = ctypes.POINTER(_Problem)
_PK, _PA, _PS = (ctypes.POINTER(t) for t in (_KVCache, _AttentionOpts, _SharedPrefix))
_sig = {
    "misa_workspace_size": (_c_sz, [_PP, _c_i32, _c_i32, _c_i32]),
    "misa_block_offsets": (ctypes.c_int, [_c_p, _c_i32, _c_i32, _c_p, _c_p]),
    "misa_pool_keys": (ctypes.c_int, [_PP, _c_p, _c_p, _c_p]),
    "misa_pool_keys_from": (ctypes.c_int, [_PP, _c_p, _c_p, _c_p, _c_p]),
    "misa_route": (ctypes.c_int, [_PP, _c_p, _c_p, _c_p, _c_p, _c_i32, _c_p, _c_p, _c_p, _c_p,
                                  _c_p, _c_sz, _c_p]),
    "misa_route_static": (ctypes.c_int, [_PP, _c_p, _c_p, _c_p, _c_p, _c_i32, _c_p, _c_p, _c_p,
                                         _c_p, _c_p]),
    "misa_score_topk": (ctypes.c_int, [_PP, _c_p, _c_p, _c_i32, _c_p, _c_i32, _c_p, _c_p, _c_p,
                                       _c_i64, _c_p, _c_sz, _c_p]),
    "misa_hier_rerank": (ctypes.c_int, [_PP, _c_p, _c_p, _c_p, _c_p, _c_i32, _c_i32, _c_p, _c_p,
                                        _c_p, _c_sz, _c_p]),
    "dsa_index_dense": (ctypes.c_int, [_PP, _c_p, _c_p, _c_p, _c_i32, _c_p, _c_p, _c_p, _c_i64,
                                       _c_p, _c_sz, _c_p]),
    "misa_stream_status": (ctypes.c_int, [_c_p, ctypes.POINTER(_c_i32)]),
    "misa_selftest_timeout": (ctypes.c_int, [_c_i32, _c_p]),
    "misa_profile_enable": (ctypes.c_int, [_c_i32]),
    "misa_profile_collect": (ctypes.c_int, [_c_i32, ctypes.c_char_p, ctypes.POINTER(ctypes.c_double),
                                            ctypes.POINTER(_c_i64)]),
    "misa_last_error_string": (ctypes.c_char_p, []),
    "misa_block_workspace_size": (_c_sz, [_PP, _c_i32]),
    "misa_block_score_topk": (ctypes.c_int, [_PP, _c_p, _c_p, _c_i32, _c_p, _c_p, _c_i32, _c_i32,
                                             _c_p, _c_p, _c_p, _c_p, _c_sz, _c_p]),
    "misa_cache_append": (ctypes.c_int, [_PP, _PK, _c_p, _c_i64, _c_p, _c_i64, _c_p, _c_i64,
                                         _c_i32, _c_p, _c_p, _c_i32, _c_i32, _c_i32, _c_p]),
    "misa_attention": (ctypes.c_int, [_PP, _PK, _c_p, _c_i32, _PA, _PS, _c_p, _c_p, _c_p, _c_sz,
                                      _c_p]),
    "misa_attention_selected": (ctypes.c_int, [_PP, _PK, _c_p, _c_i32, _PA, _c_p, _c_i32, _c_p,
                                               _c_p, _c_p, _c_sz, _c_p]),
    "misa_attention_workspace_size": (_c_sz, [_PP, _PK, _c_i32, _c_i32, _PS]),
}
for _name, (_res, _args) in _sig.items():
    _f = getattr(lib, _name)
    _f.restype, _f.argtypes = _res, _args

ERR_NAMES = {0: "OK", 1: "INVALID_ARG", 2: "UNSUPPORTED", 3: "WORKSPACE_TOO_SMALL", 4: "CUDA",
             5: "DEVICE_TIMEOUT", 6: "DEVICE_BOUNDS", 7: "DEVICE_BAD_INPUT"}


class MisaError(RuntimeError):
    def __init__(self, code: int, where: str):
        msg = lib.misa_last_error_string().decode(errors="replace")
        super().__init__(f"{where}: {ERR_NAMES.get(code, code)}: {msg}")
        self.code = code


def _check(code: int, where: str) -> None:
    if code != 0:
        raise MisaError(code, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


class Problem:
    """Shapes of one indexer call plus its device metadata.

    Built from host metadata: per-sequence key counts, per-sequence query
    counts and the query positions.  The offsets are uploaded to the device
    and block offsets are computed there by misa_block_offsets.
    """

    def __init__(self, seq_lens, query_offsets, q_pos, num_heads: int, block: int,
                 device="cuda", head_dim: int = 128, stream=None):
        import numpy as np
        import torch
        seq_lens = np.asarray(seq_lens, dtype=np.int64)
        ko = np.zeros(len(seq_lens) + 1, dtype=np.int64)
        ko[1:] = np.cumsum(seq_lens)
        self.seq_lens = seq_lens
        self.key_offsets = torch.from_numpy(ko).to(device)
        self.query_offsets = torch.from_numpy(np.asarray(query_offsets, np.int32)).to(device)
        self.q_pos = torch.from_numpy(np.asarray(q_pos, np.int32)).to(device)
        self.block_offsets = torch.empty(len(seq_lens) + 1, dtype=torch.int64, device=device)
        nblocks = int(np.sum((seq_lens + block - 1) // block))
        self.c = _Problem(
            num_seqs=len(seq_lens), num_queries=len(q_pos), num_heads=num_heads,
            head_dim=head_dim, block=block, max_seq_len=int(max(1, seq_lens.max(initial=1))),
            total_keys=int(ko[-1]), total_blocks=nblocks,
            key_offsets=self.key_offsets.data_ptr(), block_offsets=self.block_offsets.data_ptr(),
            query_offsets=self.query_offsets.data_ptr(),
            q_pos=self.q_pos.data_ptr() if len(q_pos) else None)
        block_offsets(self.key_offsets, len(seq_lens), block, self.block_offsets, stream)

    @classmethod
    def from_workload(cls, wl, device="cuda", stream=None):
        return cls(wl.seq_lens, wl.query_offsets, wl.q_pos, wl.H, wl.B, device=device,
                   head_dim=wl.d, stream=stream)

    @property
    def ref(self):
        return ctypes.byref(self.c)

    @property
    def T(self):
        return self.c.num_queries

    @property
    def H(self):
        return self.c.num_heads

    @property
    def total_blocks(self):
        return self.c.total_blocks


def workspace_size(prob: Problem, m: int, k: int, k_cand: int = 0) -> int:
    n = lib.misa_workspace_size(prob.ref, m, k, k_cand)
    if n == 0:
        raise MisaError(1, "misa_workspace_size")
    return int(n)


def block_offsets(key_offsets, num_seqs: int, block: int, out, stream=None) -> None:
    _check(lib.misa_block_offsets(_ptr(key_offsets), num_seqs, block, _ptr(out), _stream(stream)),
           "misa_block_offsets")


def pool_keys(prob: Problem, K, Kbar, stream=None) -> None:
    _check(lib.misa_pool_keys(prob.ref, _ptr(K), _ptr(Kbar), _stream(stream)), "misa_pool_keys")


def pool_keys_from(prob: Problem, K, Kbar, from_pos, stream=None) -> None:
    _check(lib.misa_pool_keys_from(prob.ref, _ptr(K), _ptr(Kbar), _ptr(from_pos),
                                   _stream(stream)), "misa_pool_keys_from")


def route(prob: Problem, q, w, K, Kbar, m: int, heads, q_r, w_r, router_scores, ws,
          stream=None) -> None:
    _check(lib.misa_route(prob.ref, _ptr(q), _ptr(w), _ptr(K), _ptr(Kbar), m, _ptr(heads),
                          _ptr(q_r), _ptr(w_r), _ptr(router_scores), _ptr(ws), ws.numel(),
                          _stream(stream)), "misa_route")


def route_static(prob: Problem, q, w, K, Kbar, m: int, heads, q_r, w_r, router_scores,
                 stream=None) -> None:
    _check(lib.misa_route_static(prob.ref, _ptr(q), _ptr(w), _ptr(K), _ptr(Kbar), m,
                                 _ptr(heads), _ptr(q_r), _ptr(w_r), _ptr(router_scores),
                                 _stream(stream)), "misa_route_static")


def score_topk(prob: Problem, q_r, w_r, m: int, K, k: int, idx, val, ws, scores_dbg=None,
               stream=None) -> None:
    ld = 0 if scores_dbg is None else scores_dbg.stride(0)
    _check(lib.misa_score_topk(prob.ref, _ptr(q_r), _ptr(w_r), m, _ptr(K), k, _ptr(idx),
                               _ptr(val), _ptr(scores_dbg), ld, _ptr(ws), ws.numel(),
                               _stream(stream)), "misa_score_topk")


def hier_rerank(prob: Problem, q, w, K, cand, k_cand: int, k: int, idx, val, ws,
                stream=None) -> None:
    _check(lib.misa_hier_rerank(prob.ref, _ptr(q), _ptr(w), _ptr(K), _ptr(cand), k_cand, k,
                                _ptr(idx), _ptr(val), _ptr(ws), ws.numel(), _stream(stream)),
           "misa_hier_rerank")


def dsa_index_dense(prob: Problem, q, w, K, k: int, idx, val, ws, scores_dbg=None,
                    stream=None) -> None:
    ld = 0 if scores_dbg is None else scores_dbg.stride(0)
    _check(lib.dsa_index_dense(prob.ref, _ptr(q), _ptr(w), _ptr(K), k, _ptr(idx), _ptr(val),
                               _ptr(scores_dbg), ld, _ptr(ws), ws.numel(), _stream(stream)),
           "dsa_index_dense")


def block_workspace_size(prob: Problem, n_blocks: int) -> int:
    n = lib.misa_block_workspace_size(prob.ref, n_blocks)
    if n == 0:
        raise MisaError(1, "misa_block_workspace_size")
    return int(n)


def block_score_topk(prob: Problem, q_r, w_r, m: int, K, Kbar, n_blocks: int, k: int, idx, val,
                     ws, blocks=None, stream=None) -> None:
    _check(lib.misa_block_score_topk(prob.ref, _ptr(q_r), _ptr(w_r), m, _ptr(K), _ptr(Kbar),
                                     n_blocks, k, _ptr(idx), _ptr(val), _ptr(blocks), _ptr(ws),
                                     ws.numel(), _stream(stream)), "misa_block_score_topk")


# ---------------------------------------------------------------- cache and attention
# These run once per layer and step, on calls of a few microseconds of GPU
# time: a check costs an attribute or two, and only a refusal builds its text.
_cuda = _raw_stream = _float32 = _int32 = None  # of torch, from the first KVCache on


def _refuse(where: str, what: str):
    raise ValueError(f"{where}: {what}")


def _token_stride(t, where: str, name: str, heads: int, dim: int, like) -> int:
    """Elements between the tokens of t, which must be [T, heads, dim] of like's dtype and
    device, the heads of a token contiguous."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        _refuse(where, f"{name} must be [T, {heads}, {dim}], got {tuple(shape)}")
    if t.dtype != like.dtype or t.device != like.device:
        _refuse(where, f"{name} must be {like.dtype} on {like.device}, got {t.dtype} on {t.device}")
    step = t.stride()
    if shape[0] and (step[2] != 1 or (heads > 1 and step[1] != dim)):
        _refuse(where, f"{name}: the heads of a token must be contiguous, got strides {step}")
    return heads * dim if shape[0] <= 1 else step[0]


def _on(cache, call, *args, stream):
    """call(*args, stream) with the cache's device current."""
    index = cache.index
    if _cuda.current_device() == index:
        return call(*args, _raw_stream(index) if stream is None else stream.cuda_stream)
    with _cuda.device(index):
        return call(*args, _raw_stream(index) if stream is None else stream.cuda_stream)


class KVCache:
    """A key/value cache for cache_append, attention and attention_selected.

    Paged: k and v [num_pages, page_size, heads, dim] views with the last axis
    contiguous (a cache that keeps its heads before its tokens is passed as
    ``x.transpose(1, 2)``), and page_table int32 [S, pages]: token p of
    sequence s is row p % page_size of page page_table[s, p // page_size].
    Packed (page_table None): k and v [total_keys, heads, dim], the tokens of
    sequence s from key_offsets[s] on, as the indexer's K.  bf16 or fp16,
    dim 64 or 128.  v None: a cache of keys only, which can be appended to.
    The tensors stay the caller's: nothing is copied, and what is written to
    the page table later counts.
    """

    def __init__(self, k, v=None, page_table=None):
        import torch
        global _cuda, _raw_stream, _float32, _int32
        _cuda, _raw_stream = torch.cuda, torch._C._cuda_getCurrentRawStream
        _float32, _int32 = torch.float32, torch.int32
        w = "KVCache"
        codes = {torch.bfloat16: 0, torch.float16: 1}
        if not k.is_cuda:
            _refuse(w, "k must be a CUDA tensor")
        if k.dtype not in codes:
            _refuse(w, f"dtype {k.dtype} unsupported (bfloat16 or float16)")
        dims = 3 if page_table is None else 4
        if k.dim() != dims or k.stride(-1) != 1:
            _refuse(w, f"k must have {dims} dimensions, the last contiguous, got {tuple(k.shape)}")
        if v is not None and (v.shape != k.shape or v.dtype != k.dtype or v.device != k.device
                              or any(n > 1 and a != b for n, a, b in zip(k.shape, k.stride(), v.stride()))):
            _refuse(w, "v must have k's shape, strides, dtype and device")
        self.k, self.v, self.page_table = k, v, page_table
        self.device, self.dtype, self.heads, self.dim = k.device, k.dtype, k.shape[-2], k.shape[-1]
        self.index = k.device.index
        c = self.c = _KVCache(k=k.data_ptr() or None, v=None if v is None else v.data_ptr() or None,
                              dtype=codes[k.dtype], num_kv_heads=self.heads, head_dim=self.dim,
                              head_stride=k.stride(-2), token_stride=k.stride(-3))
        self.seqs = None  # packed: bounded by the rows instead
        if page_table is not None:
            t = page_table
            if (t.dtype != torch.int32 or t.dim() != 2 or t.device != k.device
                    or (t.shape[1] > 1 and t.stride(1) != 1)
                    or (t.shape[0] > 1 and t.stride(0) < t.shape[1])):
                _refuse(w, "page_table must be int32 [S, pages] on the cache's device, rows contiguous "
                           "and apart (an expanded table has no room of its own for each sequence)")
            self.seqs = t.shape[0]
            c.page_size, c.num_pages, c.page_stride = k.shape[1], k.shape[0], k.stride(0)
            c.pages_per_seq = t.shape[1]
            # an empty table's address is NULL, which would mean packed; with no entries it is not read
            c.page_table = t.data_ptr() or c.k
            c.page_table_stride = max(t.stride(0), t.shape[1])
        self.ref = ctypes.byref(c)

    def _fits(self, prob: "Problem", where: str) -> None:
        if prob.q_pos.device != self.device:
            _refuse(where, f"the problem is on {prob.q_pos.device}, the cache on {self.device}")
        if self.seqs is None:
            if self.k.shape[0] < prob.c.total_keys:
                _refuse(where, f"a packed cache of {self.k.shape[0]} rows for {prob.c.total_keys} keys")
        elif self.seqs < prob.c.num_seqs:
            _refuse(where, f"a page table of {self.seqs} rows for {prob.c.num_seqs} sequences")


class SharedPrefix:
    """Sequences that begin with the same tokens: group g is sequences
    seq_offsets[g] .. seq_offsets[g+1]-1, which share their first lens[g]
    tokens.  attention reads those once, where the group's first sequence
    keeps them.  max_len bounds every length that will be written to
    ``lens`` later (default: the largest one now)."""

    def __init__(self, seq_offsets, lens, device="cuda", max_len=None):
        import numpy as np
        import torch
        so, n = np.asarray(seq_offsets, np.int32), np.asarray(lens, np.int32)
        if (so.ndim != 1 or n.ndim != 1 or len(so) != len(n) + 1 or (np.diff(so) < 0).any()
                or so[0] < 0 or (n < 0).any()):
            _refuse("SharedPrefix",
                    "needs non-decreasing seq_offsets [groups + 1] and lens [groups], all >= 0")
        self.max_len = int(n.max(initial=0)) if max_len is None else int(max_len)
        self.last = int(so[-1])
        self.seq_offsets = torch.from_numpy(so).to(device)
        self.lens = torch.from_numpy(n).to(device)
        self.c = _SharedPrefix(num_groups=len(n), max_len=self.max_len,
                               seq_offsets=self.seq_offsets.data_ptr(),
                               lens=self.lens.data_ptr() if len(n) else None)
        self.ref = ctypes.byref(self.c)


def _share_ref(share, prob, where):
    if share is None:
        return None
    if share.last > prob.c.num_seqs:
        _refuse(where, f"shared prefixes of {share.last} sequences in a batch of {prob.c.num_seqs}")
    if share.seq_offsets.device != prob.q_pos.device:
        _refuse(where, "the shared prefixes are on another device than the problem")
    return share.ref


def rope_table(rows: int, dim: int, theta: float = 10000.0, device="cuda"):
    """fp32 [rows, dim] for cache_append: cosines, then sines, of position *
    theta^(-2i/dim); angles in fp64, so that far positions keep theirs."""
    import torch
    f = theta ** (-torch.arange(0, dim, 2, dtype=torch.float64, device=device) / dim)
    a = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def cache_append(prob: Problem, cache: KVCache, k, v=None, q=None, q_out=None, rope=None,
                 interleaved: bool = False, stream=None) -> None:
    """Write the problem's query tokens' keys and values into the cache, the
    keys (and q, into q_out) rotated by their positions' rows of ``rope``."""
    w = "cache_append"
    cache._fits(prob, w)
    like, d, heads, T = cache.k, cache.dim, cache.heads, prob.T
    if (v is None) != (cache.v is None):
        _refuse(w, "v must be given exactly where the cache has values")
    if (q is None) != (q_out is None):
        _refuse(w, "q and q_out go together")
    ks = _token_stride(k, w, "k", heads, d, like)
    vs = hq = qs = rows = turned = 0
    if v is not None:
        vs = _token_stride(v, w, "v", heads, d, like)
    if q is not None:
        hq = q.shape[1] if q.dim() == 3 else 0
        qs = _token_stride(q, w, "q", hq, d, like)
        if (q_out.shape != q.shape or q_out.dtype != like.dtype or q_out.device != like.device
                or not q_out.is_contiguous()):
            _refuse(w, "q_out must be contiguous, of q's shape, dtype and device")
    if k.shape[0] != T or (v is not None and v.shape[0] != T) or (q is not None and q.shape[0] != T):
        _refuse(w, f"k, v and q must have the problem's {T} rows")
    if rope is not None:
        if (rope.dim() != 2 or rope.dtype != _float32 or rope.device != like.device
                or not rope.is_contiguous()):
            _refuse(w, "rope must be contiguous fp32 [rows, dim] on the cache's device")
        rows, turned = rope.shape
    code = _on(cache, lib.misa_cache_append, prob.ref, cache.ref, k.data_ptr(), ks,
               None if v is None else v.data_ptr(), vs, None if q is None else q.data_ptr(), qs, hq,
               None if q is None else q_out.data_ptr(), None if rope is None else rope.data_ptr(),
               rows, turned, int(interleaved), stream=stream)
    if code:
        raise MisaError(code, "misa_cache_append")


def attention_workspace_size(prob: Problem, cache: KVCache, num_q_heads: int, k: int = 0,
                             share: SharedPrefix = None) -> int:
    """Bytes of workspace of attention (k = 0) or attention_selected with lists of k."""
    with _cuda.device(cache.index):
        n = lib.misa_attention_workspace_size(prob.ref, cache.ref, num_q_heads, k,
                                              _share_ref(share, prob, "attention_workspace_size"))
    if n == 0:
        raise MisaError(1, "misa_attention_workspace_size")
    return int(n)


def _attention_args(w, prob, cache, q, out, ws, lse, scale, softcap, slopes):
    cache._fits(prob, w)
    if cache.v is None:
        _refuse(w, "the cache has no values")
    shape, dev = q.shape, cache.device
    if len(shape) != 3 or shape[0] != prob.T or shape[2] != cache.dim or not q.is_contiguous():
        _refuse(w, f"q must be contiguous [{prob.T}, heads, {cache.dim}], got {tuple(shape)}")
    if q.dtype != cache.dtype or q.device != dev:
        _refuse(w, f"q must be {cache.dtype} on {dev}, got {q.dtype} on {q.device}")
    if out.shape != shape or out.dtype != q.dtype or out.device != dev or not out.is_contiguous():
        _refuse(w, "out must be contiguous, of q's shape, dtype and device")
    if lse is not None and (lse.shape != shape[:2] or lse.dtype != _float32 or lse.device != dev
                            or not lse.is_contiguous()):
        _refuse(w, f"lse must be contiguous fp32 {tuple(shape[:2])}")
    if slopes is not None and (slopes.shape != shape[1:2] or slopes.dtype != _float32
                               or slopes.device != dev or not slopes.is_contiguous()):
        _refuse(w, f"slopes must be contiguous fp32 [{shape[1]}]")
    if ws.device != dev or not ws.is_contiguous():
        _refuse(w, "the workspace must be contiguous on the cache's device")
    opts = _AttentionOpts(cache.dim ** -0.5 if scale is None else scale, softcap,
                          None if slopes is None else slopes.data_ptr())
    return (shape[1], ctypes.byref(opts), out.data_ptr(), None if lse is None else lse.data_ptr(),
            ws.data_ptr(), ws.numel() * ws.element_size())


def attention(prob: Problem, cache: KVCache, q, out, ws, lse=None, scale=None, softcap: float = 0.0,
              slopes=None, share: SharedPrefix = None, stream=None) -> None:
    """Attention of every query over its whole prefix in the cache; a prefix
    that sequences share (``share``) is read once for all of them.  scale
    defaults to dim^-1/2; softcap caps scores by a tanh; slopes [heads]
    subtract slope * distance."""
    w = "attention"
    heads, opts, *rest = _attention_args(w, prob, cache, q, out, ws, lse, scale, softcap, slopes)
    code = _on(cache, lib.misa_attention, prob.ref, cache.ref, q.data_ptr(), heads, opts,
               _share_ref(share, prob, w), *rest, stream=stream)
    if code:
        raise MisaError(code, "misa_attention")


def attention_selected(prob: Problem, cache: KVCache, q, idx, out, ws, lse=None, scale=None,
                       softcap: float = 0.0, slopes=None, stream=None) -> None:
    """Attention of every query over the tokens idx [T, k] that an indexer
    selected for it (entries < 0 are padding)."""
    w = "attention_selected"
    heads, opts, *rest = _attention_args(w, prob, cache, q, out, ws, lse, scale, softcap, slopes)
    if (idx.dim() != 2 or idx.shape[0] != prob.T or idx.dtype != _int32
            or idx.device != cache.device or not idx.is_contiguous()):
        _refuse(w, f"idx must be contiguous int32 [{prob.T}, k] on the cache's device")
    code = _on(cache, lib.misa_attention_selected, prob.ref, cache.ref, q.data_ptr(), heads, opts,
               idx.data_ptr(), idx.shape[1], *rest, stream=stream)
    if code:
        raise MisaError(code, "misa_attention_selected")


def stream_status(stream=None) -> int:
    """Synchronise the stream; return (code, status bits) and clear the status word."""
    st = _c_i32(0)
    code = lib.misa_stream_status(_stream(stream), ctypes.byref(st))
    return code, st.value


def profile_enable(on: bool = True) -> None:
    """Bracket every library kernel launch of this thread with CUDA events."""
    lib.misa_profile_enable(1 if on else 0)


def profile_collect(max_kernels: int = 64) -> dict:
    """Synchronise and return {kernel name: (total ms, launches)}; clears the record."""
    names = ctypes.create_string_buffer(32 * max_kernels)
    ms = (ctypes.c_double * max_kernels)()
    cnt = (_c_i64 * max_kernels)()
    n = lib.misa_profile_collect(max_kernels, names, ms, cnt)
    if n < 0:
        raise MisaError(-n, "misa_profile_collect")
    out = {}
    for i in range(n):
        nm = names.raw[32 * i:32 * i + 32].split(b"\0", 1)[0].decode()
        out[nm] = (float(ms[i]), int(cnt[i]))
    return out


def selftest_timeout(wait_ms: int, stream=None) -> None:
    _check(lib.misa_selftest_timeout(wait_ms, _stream(stream)), "misa_selftest_timeout")


class Indexer:
    """Owns the device buffers of one problem and runs the call sequences.

    misa():   pool_keys -> route -> score_topk            (MISA)
    hier():   pool_keys -> route -> score_topk(k_cand) -> hier_rerank (MISA-dagger)
    dense():  dsa_index_dense                             (the DSA indexer)
    blocks(): pool_keys -> route -> block_score_topk      (routed heads x block pruning;
              needs n_blocks at construction)
    All inputs are device tensors: K uint16/bf16 [total_keys, 128],
    q [T, H, 128] bf16 bits, w [T, H] float32.
    attend(): attention over the tokens that the last of these selected.
    """

    def __init__(self, prob: Problem, m: int, k: int, k_cand: int = 0, device="cuda",
                 with_router_scores: bool = False, n_blocks: int = 0):
        import torch
        self.prob, self.m, self.k, self.k_cand = prob, m, k, k_cand
        T, H = prob.T, prob.H
        dev = device
        self.ws = torch.empty(workspace_size(prob, m, max(k, k_cand), k_cand), dtype=torch.uint8,
                              device=dev)
        self.Kbar = torch.empty((max(prob.total_blocks, 1), 128), dtype=torch.float32, device=dev)
        self.heads = torch.empty((T, m), dtype=torch.int32, device=dev)
        self.q_r = torch.empty((T, m, 128), dtype=torch.uint16, device=dev)
        self.w_r = torch.empty((T, m), dtype=torch.float32, device=dev)
        self.r = (torch.empty((T, H), dtype=torch.float32, device=dev)
                  if with_router_scores else None)
        self.idx = torch.empty((T, k), dtype=torch.int32, device=dev)
        self.val = torch.empty((T, k), dtype=torch.float32, device=dev)
        if k_cand:
            self.cand = torch.empty((T, k_cand), dtype=torch.int32, device=dev)
            self.cand_val = torch.empty((T, k_cand), dtype=torch.float32, device=dev)
        self._attend = {}
        self.n_blocks = n_blocks
        if n_blocks:
            self.block_ws = torch.empty(block_workspace_size(prob, n_blocks), dtype=torch.uint8,
                                        device=dev)
            self.blocks_kept = torch.empty((T, n_blocks), dtype=torch.int32, device=dev)

    def pool_route(self, q, w, K, stream=None, pool_from=None):
        """pool_from: None re-pools every block; else an int32 device tensor
        [S] of first new key positions (Kbar must hold the earlier blocks)."""
        if pool_from is None:
            pool_keys(self.prob, K, self.Kbar, stream)
        else:
            pool_keys_from(self.prob, K, self.Kbar, pool_from, stream)
        route(self.prob, q, w, K, self.Kbar, self.m, self.heads, self.q_r, self.w_r, self.r,
              self.ws, stream)

    def misa(self, q, w, K, stream=None, scores_dbg=None, pool_from=None):
        self.pool_route(q, w, K, stream, pool_from)
        score_topk(self.prob, self.q_r, self.w_r, self.m, K, self.k, self.idx, self.val,
                   self.ws, scores_dbg, stream)
        return self.idx, self.val

    def hier(self, q, w, K, stream=None, pool_from=None):
        self.pool_route(q, w, K, stream, pool_from)
        score_topk(self.prob, self.q_r, self.w_r, self.m, K, self.k_cand, self.cand,
                   self.cand_val, self.ws, None, stream)
        hier_rerank(self.prob, q, w, K, self.cand, self.k_cand, self.k, self.idx, self.val,
                    self.ws, stream)
        return self.idx, self.val

    def blocks(self, q, w, K, stream=None, pool_from=None):
        self.pool_route(q, w, K, stream, pool_from)
        block_score_topk(self.prob, self.q_r, self.w_r, self.m, K, self.Kbar, self.n_blocks,
                         self.k, self.idx, self.val, self.block_ws, self.blocks_kept, stream)
        return self.idx, self.val

    def dense(self, q, w, K, stream=None, scores_dbg=None):
        dsa_index_dense(self.prob, q, w, K, self.k, self.idx, self.val, self.ws, scores_dbg,
                        stream)
        return self.idx, self.val

    def attend(self, q, cache: KVCache, out=None, lse=None, scale=None, softcap: float = 0.0,
               slopes=None, stream=None):
        """Attention of q [T, heads, dim] over the tokens of the last selection
        (idx) in the key/value cache; returns out (a buffer of this object,
        written anew by the next call, unless one is given).  As the rest of this
        object its calls share buffers: on several streams they must be ordered."""
        import torch
        size = attention_workspace_size(self.prob, cache, q.shape[1], self.k)
        # kept per shape for this object's life: a captured step finds its addresses again
        key = (tuple(q.shape), q.dtype, size)
        if key not in self._attend:
            # memory of the stream that will write it: what the current one freed may still be in use there
            with torch.cuda.stream(stream):
                self._attend[key] = (torch.empty(size, dtype=torch.uint8, device=q.device),
                                     torch.empty(q.shape, dtype=q.dtype, device=q.device))
        ws, own = self._attend[key]
        out = own if out is None else out
        attention_selected(self.prob, cache, q, self.idx, out, ws, lse, scale, softcap,
                           slopes, stream)
        return out
