// Appending a step's keys and values to the cache, rotated on the way.
//
// For token t of sequence s at position p: row p of s receives v[t] and
// k[t] turned by p's angles; q_out[t] receives q[t] turned by the same.  Each
// pair (x, y) becomes (x cos - y sin, y cos + x sin), in fp32, rounded once.
// Bandwidth-bound: every element is read once and written once (32768 tokens
// of 32 + 2 * 8 heads: 167 us, 4.9 TB/s; 227 us with the loads behind the lookup).
//
// An item is 16 elements of one head (eight pairs): two 16-byte loads, two
// 16-byte stores and the pairs' eight cosines and sines, which the heads of a
// token share through L1.  A thread block takes `tokens` consecutive tokens,
// about one round of kUnroll items a thread.  What an item reads depends on its
// number alone, so its loads go out as soon as the block knows how many of its
// tokens are not padding (one load, under 0.1 us of a step of 16 x 3 tokens' 4.1), and
// the block's warps find each token's sequence, position and cache row (a chain
// of up to four loads) while they are under way.
#include "cache.cuh"

namespace misa {

bool aligned(const void* p, size_t a);                            // abi.cu
int check_ptr(const void* ptr, size_t align, const char* name);  // abi.cu

int check_batch(const misa_problem_t* p) {
  if (!p) { set_error("problem is NULL"); return MISA_ERR_INVALID_ARG; }
  if (p->num_seqs < 1 || p->num_queries < 0 || p->max_seq_len < 1 || p->total_keys < 0) {
    set_error("invalid batch sizes (S=%d T=%d max_len=%d keys=%lld)", p->num_seqs, p->num_queries,
              p->max_seq_len, (long long)p->total_keys);
    return MISA_ERR_INVALID_ARG;
  }
  if (!p->key_offsets || !p->query_offsets || (p->num_queries > 0 && !p->q_pos)) {
    set_error("problem metadata pointer is NULL");
    return MISA_ERR_INVALID_ARG;
  }
  return MISA_OK;
}

int check_cache(const misa_problem_t* p, const misa_kv_cache_t* c, bool need_v) {
  if (!c) { set_error("cache is NULL"); return MISA_ERR_INVALID_ARG; }
  if (c->dtype != MISA_BF16 && c->dtype != MISA_FP16) {
    set_error("cache dtype %d unsupported (bf16 or fp16)", c->dtype);
    return MISA_ERR_UNSUPPORTED;
  }
  if (c->head_dim != 64 && c->head_dim != 128) {
    set_error("cache head_dim %d unsupported (64 or 128)", c->head_dim);
    return MISA_ERR_UNSUPPORTED;
  }
  if (c->num_kv_heads < 1 || c->num_kv_heads > 256) {
    set_error("num_kv_heads %d outside 1..256", c->num_kv_heads);
    return MISA_ERR_INVALID_ARG;
  }
  int rc = check_ptr(c->k, 16, "cache k");
  if (!rc && need_v) rc = check_ptr(c->v, 16, "cache v");
  if (rc) return rc;
  if (c->v && !aligned(c->v, 16)) { set_error("cache v is not 16-byte aligned"); return MISA_ERR_INVALID_ARG; }
  if (c->token_stride < 0 || c->head_stride < 0 || c->token_stride % 8 || c->head_stride % 8) {
    set_error("cache strides must be non-negative multiples of 8 elements");
    return MISA_ERR_INVALID_ARG;
  }
  if (c->page_table) {
    if (!aligned(c->page_table, 4) || c->page_size < 1 || c->num_pages < 0 || c->pages_per_seq < 0 ||
        c->page_table_stride < c->pages_per_seq || c->page_stride < 0 || c->page_stride % 8) {
      set_error("invalid page table (page_size=%d pages=%d per sequence=%d stride=%lld page_stride=%lld)",
                c->page_size, c->num_pages, c->pages_per_seq, (long long)c->page_table_stride,
                (long long)c->page_stride);
      return MISA_ERR_INVALID_ARG;
    }
  }
  (void)p;
  return MISA_OK;
}

CacheView cache_view(const misa_problem_t* p, const misa_kv_cache_t* c) {
  CacheView v;
  v.k = static_cast<uint16_t*>(c->k);
  v.v = static_cast<uint16_t*>(c->v);
  v.table = c->page_table;
  v.ko = p->key_offsets;
  v.table_stride = c->page_table_stride;
  v.page_stride = c->page_stride;
  v.token_stride = c->token_stride;
  v.head_stride = c->head_stride;
  v.total_keys = p->total_keys;
  v.page_size = c->page_size > 0 ? c->page_size : 1;
  v.page_shift = -1;
  for (int b = 0; b < 31; ++b)
    if (v.page_size == (1 << b)) v.page_shift = b;
  v.num_pages = c->num_pages;
  v.pages_per_seq = c->pages_per_seq;
  return v;
}

namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 32;  // most tokens of a thread block
constexpr int kUnroll = 4;

struct AppendArgs {
  CacheView c;
  const uint16_t *k, *v, *q;
  uint16_t* q_out;
  const float* rope;
  const int32_t *qo, *q_pos;
  uint32_t* status;
  int64_t k_stride, v_stride, q_stride;
  int S, T, Hq, Hkv, D, rope_rows, rope_dim, interleaved, tokens;
  uint32_t per_magic;  // ceil(2^32 / items of a token): item number -> token by one multiplication
};

struct Pair16 {
  uint4 a, b;
};

template <typename E>
__device__ __forceinline__ void turn(Pair16& x, const float4 (&cs)[4], bool interleaved) {
  const float c[8] = {cs[0].x, cs[0].y, cs[0].z, cs[0].w, cs[1].x, cs[1].y, cs[1].z, cs[1].w};
  const float s[8] = {cs[2].x, cs[2].y, cs[2].z, cs[2].w, cs[3].x, cs[3].y, cs[3].z, cs[3].w};
  uint32_t* w[2] = {reinterpret_cast<uint32_t*>(&x.a), reinterpret_cast<uint32_t*>(&x.b)};
  const E tag = E();
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t& u = w[i >> 2][i & 3];
      const float a = to_float((uint16_t)(u & 0xffff), tag), b = to_float((uint16_t)(u >> 16), tag);
      u = pack2(a * c[i] - b * s[i], b * c[i] + a * s[i], tag);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t ua = w[0][i], ub = w[1][i];
      const float a0 = to_float((uint16_t)(ua & 0xffff), tag), a1 = to_float((uint16_t)(ua >> 16), tag);
      const float b0 = to_float((uint16_t)(ub & 0xffff), tag), b1 = to_float((uint16_t)(ub >> 16), tag);
      w[0][i] = pack2(a0 * c[2 * i] - b0 * s[2 * i], a1 * c[2 * i + 1] - b1 * s[2 * i + 1], tag);
      w[1][i] = pack2(b0 * c[2 * i] + a0 * s[2 * i], b1 * c[2 * i + 1] + a1 * s[2 * i + 1], tag);
    }
  }
}

template <typename E, int D>
__global__ void __launch_bounds__(kAppendThreads, 4) append_kernel(const __grid_constant__ AppendArgs a) {
  pdl_wait_then_release();
  __shared__ int64_t s_row[kAppendTokens];
  __shared__ int s_pos[kAppendTokens];
  const int t0 = blockIdx.x * a.tokens;
  // rows behind the last sequence's are padding, which need not be there: none is read
  const int nt = min(a.tokens, min(a.T, __ldg(a.qo + a.S)) - t0);
  if (nt <= 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kPer = D / 16;  // items of a head
  const int heads = a.Hq + a.Hkv + (a.v ? a.Hkv : 0);
  const int per_token = heads * kPer, items = nt * per_token;
  const int turned = a.rope ? a.rope_dim / 16 : 0;
  struct Where {
    int tok, h, ca, cb, pair;  // chunks of eight elements, and the angles' number or -1
  };
  auto where = [&](int it) {
    Where w;
    w.tok = (int)__umulhi((uint32_t)it, a.per_magic);
    const int in_token = it - w.tok * per_token, i = in_token % kPer;
    w.h = in_token / kPer;
    const int rot = w.h < a.Hq + a.Hkv ? turned : 0;
    // a pair's two halves, or any two chunks: eight lanes read 128 bytes together
    w.pair = i < rot ? i : -1;
    w.ca = i < rot ? i : rot + i;
    w.cb = i < rot ? i + rot : kPer + i;
    return w;
  };
  Pair16 x[kUnroll];
  auto load = [&](int base) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int it = base + u * kAppendThreads;
      if (it >= items) continue;
      const Where w = where(it);
      const int64_t t = t0 + w.tok;
      const uint16_t* src = w.h < a.Hq           ? a.q + t * a.q_stride + w.h * D
                            : w.h < a.Hq + a.Hkv ? a.k + t * a.k_stride + (w.h - a.Hq) * D
                                                 : a.v + t * a.v_stride + (w.h - a.Hq - a.Hkv) * D;
      x[u].a = __ldcs(reinterpret_cast<const uint4*>(src) + w.ca);
      x[u].b = __ldcs(reinterpret_cast<const uint4*>(src) + w.cb);
    }
  };
  load(threadIdx.x);

  for (int i = warp; i < nt; i += kAppendThreads / 32) {
    const int t = t0 + i;
    int pos = __ldg(a.q_pos + t);
    const int seq = warp_segment(a.qo, a.S, t);
    if (lane == 0) {
      const int64_t len = __ldg(a.c.ko + seq + 1) - __ldg(a.c.ko + seq);
      int64_t row = -1;
      uint32_t bad = 0;
      if (pos < 0 || pos >= len) {
        bad = MISA_STATUS_BAD_INPUT;
      } else if (a.rope && pos >= a.rope_rows) {
        bad = MISA_STATUS_BOUNDS;
      } else {
        row = cache_row(a.c, seq, pos);
        if (row < 0) bad = MISA_STATUS_BOUNDS;
      }
      if (bad) {
        set_status(a.status, bad);
        pos = -1;
      }
      s_pos[i] = pos;
      s_row[i] = row;
    }
  }
  __syncthreads();

  for (int base = threadIdx.x; base < items; base += kUnroll * kAppendThreads) {
    if (base != threadIdx.x) load(base);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int it = base + u * kAppendThreads;
      if (it >= items) continue;
      const Where w = where(it);
      const int pos = s_pos[w.tok];
      if (pos < 0) continue;
      if (w.pair >= 0) {
        const float4* c = reinterpret_cast<const float4*>(a.rope + (int64_t)pos * a.rope_dim);
        const float4* s = c + a.rope_dim / 8;
        // chunk a's and chunk b's pairs, or the eight that the two share
        const int c0 = a.interleaved ? w.ca : 2 * w.ca, c1 = a.interleaved ? w.cb : 2 * w.ca + 1;
        const float4 cs[4] = {__ldg(c + c0), __ldg(c + c1), __ldg(s + c0), __ldg(s + c1)};
        turn<E>(x[u], cs, a.interleaved != 0);
      }
      uint16_t* dst;
      if (w.h < a.Hq) {
        dst = a.q_out + ((int64_t)(t0 + w.tok) * a.Hq + w.h) * D;
      } else {
        const bool is_v = w.h >= a.Hq + a.Hkv;
        dst = (is_v ? a.c.v : a.c.k) + s_row[w.tok] + (w.h - a.Hq - (is_v ? a.Hkv : 0)) * a.c.head_stride;
      }
      *reinterpret_cast<uint4*>(dst + w.ca * 8) = x[u].a;
      *reinterpret_cast<uint4*>(dst + w.cb * 8) = x[u].b;
    }
  }
}

template <typename E>
cudaError_t launch_append(const AppendArgs& a, int blocks, cudaStream_t st) {
  return a.D == 128 ? launch_pdl(append_kernel<E, 128>, dim3(blocks), dim3(kAppendThreads), 0, st, a)
                    : launch_pdl(append_kernel<E, 64>, dim3(blocks), dim3(kAppendThreads), 0, st, a);
}

}  // namespace
}  // namespace misa

using namespace misa;

extern "C" int misa_cache_append(const misa_problem_t* p, const misa_kv_cache_t* cache, const void* k,
                                 int64_t k_stride, const void* v, int64_t v_stride, const void* q,
                                 int64_t q_stride, int32_t num_q_heads, void* q_out, const float* rope,
                                 int32_t rope_rows, int32_t rope_dim, int32_t interleaved,
                                 misa_stream_t stream) {
  int rc = check_batch(p);
  if (rc || (rc = check_cache(p, cache, false))) return rc;
  if (p->num_queries == 0) return MISA_OK;
  const int D = cache->head_dim;
  if ((v != nullptr) != (cache->v != nullptr)) {
    set_error("v and the cache's v must both be given or both be NULL");
    return MISA_ERR_INVALID_ARG;
  }
  if ((rc = check_ptr(k, 16, "k"))) return rc;
  if (v && (rc = check_ptr(v, 16, "v"))) return rc;
  const int64_t kv_row = (int64_t)cache->num_kv_heads * D;
  if (k_stride % 8 || k_stride < kv_row || (v && (v_stride % 8 || v_stride < kv_row))) {
    set_error("k_stride and v_stride must be multiples of 8 elements, at least a token's %lld",
              (long long)kv_row);
    return MISA_ERR_INVALID_ARG;
  }
  if (q) {
    if ((rc = check_ptr(q, 16, "q")) || (rc = check_ptr(q_out, 16, "q_out"))) return rc;
    if (num_q_heads < 1 || num_q_heads > 4096 || q_stride % 8 || q_stride < (int64_t)num_q_heads * D) {
      set_error("invalid q (num_q_heads=%d q_stride=%lld)", num_q_heads, (long long)q_stride);
      return MISA_ERR_INVALID_ARG;
    }
    if (q == q_out && q_stride != (int64_t)num_q_heads * D) {
      set_error("q can be rotated in place only where its rows are contiguous");
      return MISA_ERR_INVALID_ARG;
    }
  } else if (q_out) {
    set_error("q_out without q");
    return MISA_ERR_INVALID_ARG;
  }
  if (rope) {
    if ((rc = check_ptr(rope, 16, "rope"))) return rc;
    if (rope_rows < 1 || rope_dim < 16 || rope_dim % 16 || rope_dim > D) {
      set_error("rope needs rows >= 1 and a dim that is a multiple of 16, at most %d (rows=%d dim=%d)",
                D, rope_rows, rope_dim);
      return MISA_ERR_INVALID_ARG;
    }
  }
  uint32_t* status = status_ptr();
  if (!status) { set_error("status word unavailable"); return MISA_ERR_CUDA; }
  AppendArgs a;
  a.c = cache_view(p, cache);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q = static_cast<const uint16_t*>(q);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.rope = rope;
  a.qo = p->query_offsets;
  a.q_pos = p->q_pos;
  a.status = status;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_stride = q_stride;
  a.S = p->num_seqs;
  a.T = p->num_queries;
  a.Hq = q ? num_q_heads : 0;
  a.Hkv = cache->num_kv_heads;
  a.D = D;
  a.rope_rows = rope_rows;
  a.rope_dim = rope_dim;
  a.interleaved = interleaved;
  // About one round of kUnroll items per thread, but no fewer blocks than two
  // per SM while there are tokens to spread.
  const int per_token = (a.Hq + a.Hkv * (v ? 2 : 1)) * (D / 16);
  int tokens = max(1, min(kAppendTokens, kUnroll * kAppendThreads / per_token));
  tokens = max(1, min(tokens, a.T / (2 * num_sms())));
  a.tokens = tokens;
  a.per_magic = (uint32_t)(((uint64_t(1) << 32) + per_token - 1) / per_token);  // items * per_token < 2^32
  const int blocks = (a.T + tokens - 1) / tokens;
  ProfScope ps("cache_append", static_cast<cudaStream_t>(stream));
  return cuda_fail(cache->dtype == MISA_BF16
                       ? launch_append<__nv_bfloat16>(a, blocks, static_cast<cudaStream_t>(stream))
                       : launch_append<__half>(a, blocks, static_cast<cudaStream_t>(stream)),
                   "append_kernel");
}
