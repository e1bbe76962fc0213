/*
 * misa.h -- C ABI of the MISA routed sparse-attention indexer for NVIDIA B200 (sm_100a).
 *
 * Method: "MISA: Mixture of Indexer Sparse Attention for Long-Context LLM
 * Inference" (Zhou et al., 2026).  The DSA indexer scores every prefix token
 * of a query with all H indexer heads,
 *     I[t,s] = sum_h w[t,h] * ReLU(q[t,h] . k[s]),   keys s = 0..t,
 * and keeps the top-k tokens for the main attention.  MISA treats the H heads
 * as a mixture-of-experts pool: a router on mean-pooled key blocks keeps m
 * heads per query, and only those m heads run the token-level scoring.
 * MISA-dagger keeps k_cand routed candidates and re-ranks them with all H heads.
 *
 * Conventions for every entry point
 *   - All array arguments are DEVICE pointers owned by the caller; the library
 *     allocates no device memory.  Scratch space is the caller's workspace
 *     (size from misa_workspace_size).
 *   - bf16 tensors are passed as uint16_t bit patterns.  Rows are row-major
 *     and 16-byte aligned; head_dim must be 128.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *     default stream).  The return code reports argument and launch errors
 *     only.  Device-side conditions (a bounded wait that timed out, an index
 *     out of range, a position or candidate out of its sequence) set bits in
 *     a per-device status word read by misa_stream_status.
 *   - No call throws; on error the message is kept in a thread-local buffer
 *     (misa_last_error_string).
 *   - Ties: heads are ranked by (router score desc, head index asc); tokens by
 *     (score desc, token index asc); -0 counts as +0.  A query whose prefix is
 *     shorter than k selects every prefix token and pads its row with index
 *     -1 and value -inf.  Row order of idx/val is unspecified.
 *   - NaN (from a NaN in q, w or K): a head whose router score is NaN is
 *     ranked last and MISA_STATUS_BAD_INPUT is set; a NaN token score ranks
 *     below every number, so it is selected only when its row has fewer
 *     other scores than min(k, prefix length), and then (with value NaN)
 *     the same bit is set.
 */
#ifndef MISA_H_
#define MISA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef void* misa_stream_t; /* cudaStream_t */

/* Return codes. */
enum {
  MISA_OK = 0,
  MISA_ERR_INVALID_ARG = 1,        /* null pointer, bad size, misaligned pointer */
  MISA_ERR_UNSUPPORTED = 2,        /* valid but not built: head_dim != 128, m not a power of two ... */
  MISA_ERR_WORKSPACE_TOO_SMALL = 3,
  MISA_ERR_CUDA = 4,               /* a CUDA runtime call failed (message has the CUDA error) */
  MISA_ERR_DEVICE_TIMEOUT = 5,     /* misa_stream_status only */
  MISA_ERR_DEVICE_BOUNDS = 6,      /* misa_stream_status only */
  MISA_ERR_DEVICE_BAD_INPUT = 7    /* misa_stream_status only */
};

/* Bits of the device status word. */
#define MISA_STATUS_TIMEOUT   0x1u /* a bounded wait in a kernel gave up; that CTA returned early */
#define MISA_STATUS_BOUNDS    0x2u /* an index fell outside its buffer; the access was skipped */
#define MISA_STATUS_BAD_INPUT 0x4u /* a query position or candidate outside its sequence, a NaN
                                      router score, or a NaN token score in a selection */

/*
 * Problem description (the shapes of one indexer call).
 *
 * Keys of all sequences are packed: K is [total_keys, head_dim] bf16 and
 * sequence s owns rows key_offsets[s] .. key_offsets[s+1]-1.  Its pooled keys
 * (one per block of `block` consecutive keys, the last block possibly
 * partial) are rows block_offsets[s] .. block_offsets[s+1]-1 of Kbar, with
 * block_offsets[s+1]-block_offsets[s] = ceil(L_s / block)  (gist.science
 * summary, "Methodologie: MISA": M = ceil(L/B) blocks).  Queries of sequence
 * s are rows query_offsets[s] .. query_offsets[s+1]-1 of q / w; query t sits
 * at position q_pos[t] in its sequence and sees keys 0..q_pos[t] (causal,
 * self included).
 */
typedef struct {
  int32_t num_seqs;              /* S >= 1 */
  int32_t num_queries;           /* T >= 0 */
  int32_t num_heads;             /* H, 1..64 */
  int32_t head_dim;              /* d, must be 128 */
  int32_t block;                 /* B, pooling block, 1..4096 */
  int32_t max_seq_len;           /* host-side upper bound on every L_s (sizes grids) */
  int64_t total_keys;            /* rows of K = key_offsets[S] */
  int64_t total_blocks;          /* rows of Kbar = block_offsets[S] */
  const int64_t* key_offsets;    /* device [S+1], non-decreasing, key_offsets[0] = 0 */
  const int64_t* block_offsets;  /* device [S+1], see misa_block_offsets */
  const int32_t* query_offsets;  /* device [S+1], non-decreasing, query_offsets[0] = 0 */
  const int32_t* q_pos;          /* device [T], 0 <= q_pos[t] < L_seq(t) */
} misa_problem_t;

/* Bytes of workspace that any entry point below needs for this problem with
 * m routed heads, final top-k `k` and MISA-dagger candidate count `k_cand`
 * (0 if unused), on its fastest path.  Returns 0 on invalid arguments.
 * For a prefill that streams (misa_score_topk, dsa_index_dense) this
 * includes candidate lists per query row for the exact selection after the
 * scoring pass, about T * (2 * 1.4 * k / 128 + 16) KB with that row count
 * between 32 and 256 (8.1 GB for 131072 queries at k = 2048, 25 GB at the
 * MISA-dagger keep k = 8192); a smaller workspace takes slower paths (selection
 * inside the scoring kernel, then score rows with a separate top-k) and
 * MISA_ERR_WORKSPACE_TOO_SMALL only below what the slowest path needs. */
size_t misa_workspace_size(const misa_problem_t* p, int32_t m, int32_t k, int32_t k_cand);

/* block_offsets[s] = sum_{s'<s} ceil(L_s' / block) from key_offsets
 * (device arrays, S+1 entries each). */
int misa_block_offsets(const int64_t* key_offsets, int32_t num_seqs, int32_t block,
                       int64_t* block_offsets, misa_stream_t stream);

/* Step 1 -- mean-pooled keys (gist.science summary, "Methodologie: MISA",
 * Lightweight Block-Pooled Router: mean-pooled indexer keys per block).
 * Kbar[b,:] = (1/|b|) sum_{s in b} K[s,:], the last block of a sequence
 * averaged over the keys present.  Summed in fp64, divided in fp64, rounded
 * once to fp32.
 *   K    [total_keys, 128] bf16;  Kbar [total_blocks, 128] fp32 (written). */
int misa_pool_keys(const misa_problem_t* p, const uint16_t* K, float* Kbar, misa_stream_t stream);

/* Step 1, incremental (decode): re-pools only the blocks of each sequence s
 * that hold keys at positions >= from_pos[s] (e.g. the keys appended since
 * Kbar was last computed); every other row of Kbar is left unchanged, so
 * Kbar must already hold the pooled means of the earlier blocks.  Same
 * arithmetic as misa_pool_keys, so the updated rows are bit-identical to a
 * full re-pooling.
 *   from_pos [S] int32 device array; a value <= 0 re-pools the whole
 *   sequence, a value >= its length leaves it unchanged.  One CTA per
 *   sequence. */
int misa_pool_keys_from(const misa_problem_t* p, const uint16_t* K, float* Kbar,
                        const int32_t* from_pos, misa_stream_t stream);

/* Step 2 -- block-pooled router (same passage: per-head affinities on the
 * pooled keys, aggregated into one importance score per head, top-h heads).
 *     r[t,h] = w[t,h] * sum_{b < M_t} ReLU(q[t,h] . Kbar_t[b]),  M_t = ceil((t+1)/B)
 * over the floor((t+1)/B) full blocks of Kbar plus, when (t+1) mod B != 0,
 * the causal partial block (mean of keys floor((t+1)/B)*B .. t).  Keeps the
 * m best heads per query.
 *   q [T, H, 128] bf16;  w [T, H] fp32;  K, Kbar as above;  1 <= m <= H, m a power of two.
 *   heads [T, m] int32  (written; rank order);
 *   q_r   [T, m, 128] bf16 (written; q_r[t,j] = q[t, heads[t,j]]);
 *   w_r   [T, m] fp32  (written; w_r[t,j] = w[t, heads[t,j]]);
 *   router_scores [T, H] fp32 or NULL (written if not NULL). */
int misa_route(const misa_problem_t* p, const uint16_t* q, const float* w, const uint16_t* K,
               const float* Kbar, int32_t m, int32_t* heads, uint16_t* q_r, float* w_r,
               float* router_scores, void* ws, size_t ws_bytes, misa_stream_t stream);

/* misa_route without a caller workspace: its scratch is a fixed 4 MiB device
 * array inside the library (one per device), for callers that cannot
 * allocate on the decode path (a host runtime with no device allocator of
 * its own, or code that must not call cudaMalloc there).  No counterpart in
 * the paper.  Arguments and results as misa_route, which it runs with that
 * array as its workspace; it allocates no memory.
 *   - The first call on each device (with that device current) looks up the
 *     array's address; make it before capturing a stream that uses the call.
 *   - Nothing in the array needs to start at zero.
 *   - Calls on one device must not overlap in execution: they share the
 *     array and race on it.  Issue them on one stream, or order them.
 *   - MISA_ERR_UNSUPPORTED when the problem needs more than 4 MiB of router
 *     scratch (the message gives both sizes): decode batches fit; prefill
 *     fits up to about 7K keys, since the tensor-core router keeps a 512-byte
 *     running block mean per key.  MISA_ERR_INVALID_ARG while tracing is on
 *     for the calling thread. */
int misa_route_static(const misa_problem_t* p, const uint16_t* q, const float* w,
                      const uint16_t* K, const float* Kbar, int32_t m, int32_t* heads,
                      uint16_t* q_r, float* w_r, float* router_scores, misa_stream_t stream);

/* Steps 3+4 -- routed token scoring and per-query top-k (same section,
 * Sparse Token Scoring: only the routed heads score the full prefix; the
 * top-k tokens come from these reduced scores).
 *     I[t,s] = sum_{j<m} w_r[t,j] * ReLU(q_r[t,j] . K[s]),  s = 0..q_pos[t]
 *   q_r [T, m, 128] bf16;  w_r [T, m] fp32;  1 <= k <= 65536.
 *   idx [T, k] int32 token indices within the sequence;  val [T, k] fp32 scores.
 *   scores_dbg: NULL, or [T, scores_ld] fp32 receiving I[t, 0..q_pos[t]]
 *   (entries past the prefix are unspecified); scores_ld >= max_seq_len. */
int misa_score_topk(const misa_problem_t* p, const uint16_t* q_r, const float* w_r, int32_t m,
                    const uint16_t* K, int32_t k, int32_t* idx, float* val, float* scores_dbg,
                    int64_t scores_ld, void* ws, size_t ws_bytes, misa_stream_t stream);

/* Step 5 -- MISA-dagger fine stage (gist.science summary, "Hierarchische
 * Variant (MISA†)"): the all-head DSA indexer re-scores only the candidate
 * tokens and keeps the final top-k.
 *   cand [T, k_cand] int32 token indices (e.g. the idx of misa_score_topk
 *   run with k = k_cand); entries < 0 are padding and skipped; an entry past
 *   the query's position sets MISA_STATUS_BAD_INPUT and is skipped.
 *   idx [T, k], val [T, k] as in misa_score_topk;  k <= k_cand <= 65536. */
int misa_hier_rerank(const misa_problem_t* p, const uint16_t* q, const float* w,
                     const uint16_t* K, const int32_t* cand, int32_t k_cand, int32_t k,
                     int32_t* idx, float* val, void* ws, size_t ws_bytes, misa_stream_t stream);

/* Head axis x token axis -- routed heads with block pruning.  The heads the
 * router kept (q_r, w_r of misa_route) first score the pooled key blocks,
 *     S[t,b] = sum_{j<m} w_r[t,j] * ReLU(q_r[t,j] . Kbar[b]),
 * over the full blocks b < floor((q_pos[t]+1)/B) of the query's sequence;
 * the n_blocks best blocks by (S desc, block asc) are kept (HISA abstract on
 * the thelatestinai.com papers page: a block-level coarse filter on pooled
 * block representations, then token-level refinement inside the kept
 * blocks; gist.science summary of the MISA paper, "Betekenis en Claims":
 * head-axis routing combines with token-level schemes).  The candidates are
 * the keys of the kept blocks plus the keys floor((q_pos[t]+1)/B)*B ..
 * q_pos[t] of the query's own incomplete block; the routed heads score them
 * (as misa_score_topk does the whole prefix) and the top-k is kept.  A query
 * with fewer than n_blocks full blocks keeps them all, so with n_blocks >=
 * ceil(max_seq_len / B) the result is misa_score_topk's.
 *   q_r [T, m, 128] bf16, w_r [T, m] fp32 (from misa_route); K; Kbar
 *   (misa_pool_keys); m a power of two <= min(64, H);
 *   n_blocks >= 1 with (n_blocks + 1) * B <= 65536;
 *   1 <= k <= (n_blocks + 1) * B;
 *   idx [T, k] int32, val [T, k] fp32 as in misa_score_topk;
 *   blocks: NULL, or [T, n_blocks] int32 receiving the kept block indices
 *   within the sequence (row order unspecified, -1 padding);
 *   ws: misa_block_workspace_size(p, n_blocks) bytes, 256-byte aligned.
 * Five launches on `stream` (block scores, block top-k, candidate
 * expansion, candidate scoring, top-k); no host synchronisation. */
size_t misa_block_workspace_size(const misa_problem_t* p, int32_t n_blocks);
int misa_block_score_topk(const misa_problem_t* p, const uint16_t* q_r, const float* w_r,
                          int32_t m, const uint16_t* K, const float* Kbar, int32_t n_blocks,
                          int32_t k, int32_t* idx, float* val, int32_t* blocks, void* ws,
                          size_t ws_bytes, misa_stream_t stream);

/* The dense DSA indexer, the in-run comparison (MISA abstract; gist.science
 * summary, "Probleemstelling"): every head scores every prefix token.
 *     I[t,s] = sum_{h<H} w[t,h] * ReLU(q[t,h] . K[s])
 * Same outputs as misa_score_topk; H must be a power of two. */
int dsa_index_dense(const misa_problem_t* p, const uint16_t* q, const float* w,
                    const uint16_t* K, int32_t k, int32_t* idx, float* val, float* scores_dbg,
                    int64_t scores_ld, void* ws, size_t ws_bytes, misa_stream_t stream);

/* ------------------------------------------------------------------------
 * The key/value cache around the indexer: writing a step's keys and values
 * into it, and attending over it -- over every token, or over the tokens
 * that the indexer selected (gist.science summary, "Probleemstelling": the
 * indexer's top-k tokens are what the main attention then reads).
 *
 * These calls read from misa_problem_t the batch only (num_seqs,
 * num_queries, max_seq_len, total_keys, key_offsets, query_offsets, q_pos);
 * num_heads, head_dim, block, total_blocks and block_offsets belong to the
 * indexer and may hold anything.  L_s = key_offsets[s+1] - key_offsets[s]
 * tokens of sequence s are in the cache, the queries' own included.  Query
 * rows at and behind query_offsets[S] are padding: nothing of theirs is read
 * and their rows of every output are left as they were.
 * ------------------------------------------------------------------------ */
enum { MISA_BF16 = 0, MISA_FP16 = 1 };

/* A cache of keys and values, num_kv_heads heads of head_dim elements a token.
 *   Paged (page_table != NULL): token p of sequence s is row p % page_size of
 *   page page_table[s * page_table_stride + p / page_size]; its head h starts
 *       page * page_stride + (p % page_size) * token_stride + h * head_stride
 *   elements behind k (and behind v).  Any order of pages, any page size, and
 *   either order of tokens and heads in a page (the strides say which).
 *   Packed (page_table == NULL): token p of sequence s is row
 *   key_offsets[s] + p, token_stride elements apart: the layout of the
 *   indexer's K.  page_size, num_pages, pages_per_seq and page_stride are
 *   not read.
 * k and v are 16-byte aligned; strides are multiples of 8 elements.  A page
 * number outside 0..num_pages-1, or a token past pages_per_seq * page_size
 * (past total_keys, packed), sets MISA_STATUS_BOUNDS and is skipped.
 * Attention over many rows a key head runs on the 5th-generation tensor cores
 * where the greatest common divisor of the strides (of axes longer than one) is
 * at least head_dim and the cache spans fewer than 2^31 such steps; any other
 * layout, such as pages a few elements apart, gives the same results by the
 * warp-level kernel: 2 x 1000 queries behind 16384 tokens in 2.2 ms, not 0.5. */
typedef struct {
  void* k;
  void* v;                       /* NULL: keys only (misa_cache_append) */
  int32_t dtype;                 /* MISA_BF16 or MISA_FP16 */
  int32_t num_kv_heads;          /* 1..256 */
  int32_t head_dim;              /* 64 or 128 */
  int32_t page_size;             /* tokens of a page, >= 1 */
  int32_t num_pages;             /* pages behind k */
  int32_t pages_per_seq;         /* entries of a sequence's row of page_table */
  const int32_t* page_table;     /* device [S, page_table_stride], or NULL */
  int64_t page_table_stride;
  int64_t page_stride, token_stride, head_stride;  /* elements */
} misa_kv_cache_t;

/* What happens to a product before the softmax:
 *     x = scale * (q . k[s]);   softcap > 0: x = softcap * tanh(x / softcap);
 *     slopes != NULL: x -= slopes[head] * (q_pos[t] - s).
 * An x of -inf counts as masked; a NaN reaches the row's output, and no other
 * row's.  A cap puts x off by at most 3 2^-20 |x|, however large it is: one far
 * above the scores is as none. */
typedef struct {
  float scale;
  float softcap;                 /* 0: none, else any finite value > 0 */
  const float* slopes;           /* device fp32 [num_q_heads], or NULL */
} misa_attention_opts_t;

/* Sequences that begin with the same tokens: those of group g are
 * seq_offsets[g] .. seq_offsets[g+1]-1, and their first lens[g] tokens are
 * read once for all of them, at the place where the group's first sequence
 * keeps them (a length below 0, beyond that sequence's own or beyond max_len
 * sets MISA_STATUS_BAD_INPUT and is cut; with max_len 0 no length is read).
 * A sequence in no group shares nothing; the length of a group without
 * sequences is not looked at. */
typedef struct {
  int32_t num_groups;            /* >= 0 */
  int32_t max_len;               /* host-side upper bound on every length */
  const int32_t* seq_offsets;    /* device [num_groups + 1], non-decreasing, within 0..S */
  const int32_t* lens;           /* device [num_groups] */
} misa_shared_prefix_t;

/* Writes the keys and values of the problem's query tokens into the cache,
 * with the rotation of their position applied on the way: token t of
 * sequence s lands at token q_pos[t] of s.
 *   k, v: [T, num_kv_heads, head_dim] of the cache's type, tokens
 *   k_stride / v_stride elements apart (slices of a fused projection need no
 *   copy), heads head_dim apart; v NULL exactly where cache->v is.
 *   q: NULL, or [T, num_q_heads, head_dim], tokens q_stride apart; q_out
 *   receives its rotated rows, contiguous.  q_out may be q itself where
 *   q_stride = num_q_heads * head_dim; no other overlap is allowed.
 *   rope: NULL (nothing is rotated), or fp32 [rope_rows, rope_dim], row p the
 *   cosines of position p, then its sines, rope_dim / 2 each.  The first
 *   rope_dim elements of a head are rotated, the rest copied; pair i is
 *   elements (i, i + rope_dim / 2), or (2i, 2i + 1) with `interleaved`:
 *       (x, y) -> (x cos - y sin, y cos + x sin)
 *   in fp32, rounded once.  rope_dim: a multiple of 16, at most head_dim.
 * A position outside its sequence sets MISA_STATUS_BAD_INPUT, one past
 * rope_rows MISA_STATUS_BOUNDS; that token is left out, its q_out row too.
 * Two tokens at one position of one sequence race for its row. */
int misa_cache_append(const misa_problem_t* p, const misa_kv_cache_t* cache, const void* k,
                      int64_t k_stride, const void* v, int64_t v_stride, const void* q,
                      int64_t q_stride, int32_t num_q_heads, void* q_out, const float* rope,
                      int32_t rope_rows, int32_t rope_dim, int32_t interleaved,
                      misa_stream_t stream);

/* Attention of every query over tokens 0..q_pos[t] of its sequence:
 *     out[t,h] = sum_s softmax_s(x[t,h,s]) v[s, h / (num_q_heads / num_kv_heads)]
 *   q, out [T, num_q_heads, head_dim] of the cache's type, contiguous, no
 *   overlap;
 *   num_q_heads a multiple of num_kv_heads, at most 64 times as many heads
 *   per key head; lse: NULL, or fp32 [T, num_q_heads] receiving
 *   ln sum_s exp(x).  A query that sees no token (a position outside its
 *   sequence, flagged MISA_STATUS_BAD_INPUT; every x masked) gets a row of
 *   zeros and an lse of -inf.
 *   share: NULL, or the sequences' common prefixes.
 *   ws: misa_attention_workspace_size(p, cache, num_q_heads, 0, share) bytes,
 *   256-byte aligned; contents need not be kept or cleared.  Calls that may
 *   run at the same time need workspaces of their own.
 * Products and sums in fp32; the softmax weights enter the second product
 * rounded to the cache's type, their sum does not.  The same inputs give the
 * same bits. */
int misa_attention(const misa_problem_t* p, const misa_kv_cache_t* cache, const void* q,
                   int32_t num_q_heads, const misa_attention_opts_t* opts,
                   const misa_shared_prefix_t* share, void* out, float* lse, void* ws,
                   size_t ws_bytes, misa_stream_t stream);

/* Attention of every query over the tokens that an indexer selected for it:
 * as misa_attention, with s running over idx[t, 0..k-1] (misa_score_topk and
 * its relatives write it) instead of the whole prefix.
 *   idx [T, k] int32 token indices within the sequence, any order; entries
 *   < 0 are padding; one past the query's position sets
 *   MISA_STATUS_BAD_INPUT and is skipped; a token listed twice counts twice.
 *   1 <= k <= 65536.  ws: misa_attention_workspace_size(p, cache,
 *   num_q_heads, k, NULL) bytes. */
int misa_attention_selected(const misa_problem_t* p, const misa_kv_cache_t* cache, const void* q,
                            int32_t num_q_heads, const misa_attention_opts_t* opts,
                            const int32_t* idx, int32_t k, void* out, float* lse, void* ws,
                            size_t ws_bytes, misa_stream_t stream);

/* Bytes of workspace of misa_attention (k = 0) or misa_attention_selected
 * (k >= 1, share NULL).  Never 0 for valid arguments; 0 on invalid ones. */
size_t misa_attention_workspace_size(const misa_problem_t* p, const misa_kv_cache_t* cache,
                                     int32_t num_q_heads, int32_t k,
                                     const misa_shared_prefix_t* share);

/* Synchronises `stream`, returns the status word of the current device in
 * *device_status (may be NULL) and clears it.  Returns MISA_OK when the word
 * was zero, else the MISA_ERR_DEVICE_* code of its lowest set bit;
 * MISA_ERR_CUDA if the synchronisation itself failed. */
int misa_stream_status(misa_stream_t stream, int32_t* device_status);

/* Diagnostic: launches one CTA whose bounded wait on a barrier that nothing
 * arrives on runs out after `wait_ms` milliseconds (1..5000); the kernel then
 * sets MISA_STATUS_TIMEOUT and returns.  Used to test that a timed-out wait
 * leaves the context usable.  No counterpart in the paper. */
int misa_selftest_timeout(int32_t wait_ms, misa_stream_t stream);

/* Tracing.  While enabled (on != 0), every kernel the library launches from
 * the calling host thread is bracketed by CUDA events recorded on its launch
 * stream.  misa_profile_collect synchronises those events and returns, per
 * traced name (names: max_kernels x 32 chars), the summed device time in
 * milliseconds and the number of kernels launched under it (one per name,
 * except "plan_groups" for plans of more than 256 query groups: a scan and a
 * fill), then clears the record.  Returns the
 * number of kernel names (at most max_kernels) or a negative MISA_ERR code.
 * Names starting with '#' are counters, not kernels (time 0, the count in
 * `launches`): "#rescan_queries" sums, over the streaming top-k calls traced,
 * the queries whose sampled threshold did not hold and were rescanned.
 * While tracing, each such call also queues a 4-byte device-to-host copy
 * into pinned host memory the library keeps for this purpose.
 * No counterpart in the paper. */
int misa_profile_enable(int32_t on);
int misa_profile_collect(int32_t max_kernels, char* names, double* total_ms, int64_t* launches);

/* Message of the last failed call on this host thread ("" if none). */
const char* misa_last_error_string(void);

#ifdef __cplusplus
}
#endif

#endif /* MISA_H_ */
