// Attention over the key/value cache for many rows per key head (prefill, a
// prefix shared by a batch, a selection read by many heads) on the
// 5th-generation tensor cores.
//
//     S = Q K^T,  P = 2^(x(S) - m),  O += P V        (128 rows x 128 keys a step)
// Each block runs two streams, A and B, of 128 rows each, so that one stream's
// softmax overlaps the other's matrix products:
//   pair   A and B are different rows against the same key tiles;
//   split  A and B are the same rows against alternate key tiles, joined at
//          the end (at most 128 rows a unit, or a selection, whose keys are
//          one query's own).
// TMEM holds S_A, S_B, O_A, O_B (fp32, 128 columns each).  P overwrites the
// first half of its S in the cache's type and is the A operand of the second
// product straight from there; V [keys][dims] is its B operand as it lies
// (N-major).  A row is a TMEM lane is a thread: maximum and sum need no
// exchange.  O is rescaled only when a row's maximum has grown by more than
// 2^8 since its reference was taken (the result does not depend on the
// reference), which after the first tiles hardly happens.
//
// Warps 0-3 gather key and value rows by cp.async into a ring of 128-row
// tiles, 128-byte swizzled; warps 4-7 and 8-11 are the softmax of A and B;
// warp 12 issues the products (one thread).  Blocks are persistent; the
// gathering warps run ahead into the next item.
#include <type_traits>

#include "attend.cuh"

namespace misa {
namespace {

constexpr int kTcThreads = 512;
constexpr int kTile = 128;          // keys of a tile, rows of a stream
constexpr float kSlack = 8.f;       // log2 of how far a row's maximum may outgrow its reference
constexpr int kKeep = 8;            // tiles whose key masks are kept

template <int D, bool PAIR>
struct Tc {
  static constexpr int halves = D / 64;
  static constexpr int half = kTile * 128;                 // 64 dims of a tile
  static constexpr int tile = half * halves;
  static constexpr int q_tiles = PAIR ? 2 : 1;
  static constexpr int slots = D == 128 ? 5 : 10;
  static constexpr int off_ring = q_tiles * tile;
  static constexpr int off_key = off_ring + slots * tile;  // positions, selected mode with a bias
  static constexpr int off_inv = off_key + (PAIR ? 0 : kKeep * kTile * 4);
  static constexpr int off_ml = off_inv + kKeep * 16;
  static constexpr int off_bar = off_ml + (PAIR ? 0 : 2 * kTile * 8);
  static constexpr int bars = 2 * slots + 9;
  static constexpr int off_sum = off_bar + bars * 8;
  static constexpr int bytes = off_sum + 16 + (kScan + 1 + kScan / 32) * 4 + 1024;
};

template <typename E>
__host__ __device__ constexpr uint32_t tc_idesc(int N, bool b_mn) {
  const uint32_t f = sizeof(E) == 2 && std::is_same<E, __nv_bfloat16>::value ? 1u : 0u;
  return (1u << 4) | (f << 7) | (f << 10) | (b_mn ? 1u << 16 : 0u) | (uint32_t(N >> 3) << 17) |
         (uint32_t(kTile >> 4) << 24);
}

// V as the B operand: dims contiguous (N-major), 128-byte swizzle: atoms of
// 64 dims x 8 keys, 1024 bytes; eight keys on, 1024 bytes; 64 dims on, a half.
__device__ __forceinline__ uint64_t sw128_nmajor_desc(uint32_t addr, uint32_t half) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(half >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32],"
      " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]),
      "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// What every role works out for itself about an item.
struct Span {
  Item it;
  int k0, k1, n;  // keys, and tiles of them
  int near;       // every row that sees anything sees the keys up to this one
  bool live;
};

template <int MODE, int ROWS>
__device__ __forceinline__ Span span_of(const AttendArgs& a, const int* sums, int64_t w) {
  Span s;
  const int lane = threadIdx.x & 31;
  s.live = true;
  s.near = 0x7fffffff;
  s.it.h = (int)(w % a.Hkv);
  if constexpr (MODE == kSelected) {
    s.live = find_selected(a, ROWS, (int)(w / a.Hkv), s.it);
    s.k0 = s.it.k0;
    s.k1 = s.it.k1;
    if (s.live) {
      const int pos = __ldg(a.q_pos + s.it.qb);
      if (pos < 0 || pos >= seq_len(a, s.it.seq)) s.k1 = s.k0;  // sees nothing
    }
  } else {
    find_item<MODE>(a, ROWS, sums, (int)(w / a.Hkv), s.it);
    s.k0 = s.it.k0;
    s.k1 = s.it.k1;
    const int q0 = s.it.qb + s.it.r0 / a.G, q1 = s.it.qb + (s.it.r0 + s.it.nrows - 1) / a.G;
    const int len = MODE == kOwn ? seq_len(a, s.it.seq) : 0x7fffffff;
    int far = -1;
    for (int t = q0 + lane; t <= q1; t += 32) {
      const int pos = __ldg(a.q_pos + t);
      if (pos >= 0 && pos < len) {
        far = max(far, pos);
        s.near = min(s.near, pos);
      }
    }
    s.near = __reduce_min_sync(0xffffffffu, s.near);
    // no key behind the furthest query of the item
    if constexpr (MODE == kOwn) s.k1 = min(s.k1, __reduce_max_sync(0xffffffffu, far) + 1);
  }
  s.n = s.live && s.k1 > s.k0 ? (s.k1 - s.k0 + kTile - 1) / kTile : 0;
  return s;
}

// Order of the ring.  pair: K0 V0 K1 V1 ..; split: K0 K1 V0 K2 V1 K3 .. V(n-1).
template <bool PAIR>
__device__ __forceinline__ int place_k(int t) { return PAIR ? 2 * t : (t == 0 ? 0 : 2 * t - 1); }
template <bool PAIR>
__device__ __forceinline__ int place_v(int t, int n) { return PAIR ? 2 * t + 1 : (t == n - 1 ? 2 * n - 1 : 2 * t + 2); }

template <typename E, int D, int MODE, bool PAIR, bool PLAIN>
__global__ void __launch_bounds__(kTcThreads, 1) attend_tc_kernel(const __grid_constant__ AttendArgs a) {
  pdl_wait_then_release();
  using L = Tc<D, PAIR>;
  constexpr int kRows = kTile * L::q_tiles;
  constexpr int kSlots = L::slots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + L::off_ring;
  int* s_key = reinterpret_cast<int*>(smem + L::off_key);
  uint32_t* s_inv = reinterpret_cast<uint32_t*>(smem + L::off_inv);
  float2* s_ml = reinterpret_cast<float2*>(smem + L::off_ml);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::off_bar);
  uint64_t* empty = full + kSlots;
  uint64_t* s_full = empty + kSlots;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* q_full = o_full + 2;
  uint64_t* ml_full = q_full + 1;
  uint64_t* drain = ml_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::off_sum);
  int* abort = reinterpret_cast<int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  volatile int* s_cut = abort + 1;  // something was cut out of a value tile of this block
  int* s_sum = abort + 3;
  int total;
  if constexpr (MODE == kSelected) {
    total = a.T * ((a.G + kRows - 1) / kRows) * a.nch_max;
  } else {
    total = count_items<MODE>(a, kRows, s_sum);
  }
  const int64_t items = (int64_t)total * a.Hkv;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&full[i], 4);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(q_full, 8);
    mbar_init(ml_full, 8);
    mbar_init(drain, 1);
    *abort = 0;
    *s_cut = 0;
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 4) {
    // ------------------------------------------------------------ gathering
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    constexpr int kChunks = D / 8, kPer = 32 / kChunks;
    const int c = lane % kChunks, sub = lane / kChunks;
    int cnt = 0, told = 0;  // tiles issued and announced
    int seen = 0;           // key tiles of the items before
    bool ok = true;
    auto announce = [&](int upto) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0)
        for (; told < upto; ++told) mbar_arrive(&full[told % kSlots]);
      told = upto;
    };
    for (int64_t w = blockIdx.x; ok && w < items; w += gridDim.x) {
      const Span s = span_of<MODE, kRows>(a, s_sum, w);
      if (s.n == 0) continue;
      const int64_t head = s.it.h * a.c.head_stride;
      const int pos = MODE == kSelected ? __ldg(a.q_pos + s.it.qb) : 0;
      // lane l knows key 32 warp + l of a tile
      auto key_of = [&](int t) -> int {
        const int j = s.k0 + t * kTile + warp * 32 + lane;
        if (t >= s.n || j >= s.k1) return -1;
        return MODE == kSelected ? __ldg(a.idx + (int64_t)s.it.qb * a.k + j) : j;
      };
      auto row_of = [&](int key) -> int64_t {
        if (key < 0) return -1;
        if (MODE == kSelected && key > pos) {
          set_status(a.status, MISA_STATUS_BAD_INPUT);
          return -1;
        }
        const int64_t r = cache_row(a.c, s.it.seq, key);
        if (r < 0) set_status(a.status, MISA_STATUS_BOUNDS);
        return r;
      };
      int key_cur = key_of(0), key_next = key_of(1);
      int64_t row_prev = -1, row_cur = row_of(key_cur);
      int t_k = 0;  // next tile whose keys are loaded
      for (int m = 0; m < 2 * s.n; ++m) {
        bool is_k;
        int t;
        if (PAIR) {
          is_k = (m & 1) == 0;
          t = m >> 1;
        } else {
          is_k = m == 0 || ((m & 1) && (m + 1) / 2 < s.n);
          t = is_k ? (m + 1) / 2 : (m == 2 * s.n - 1 ? s.n - 1 : (m - 2) / 2);
        }
        const int slot = cnt % kSlots;
        if (!__all_sync(0xffffffffu, mbar_try_wait(&empty[slot], ((cnt / kSlots) & 1) ^ 1))) {
          cp_async_wait_group<0>();  // what has been issued is announced before waiting
          announce(cnt);
          if (!warp_wait(&empty[slot], ((cnt / kSlots) & 1) ^ 1, abort, a.status)) { ok = false; break; }
        }
        int64_t row;
        if (is_k) {
          if (t_k > 0) {
            row_prev = row_cur;
            key_cur = key_next;
            row_cur = row_of(key_cur);
            key_next = key_of(t + 1);
          }
          ++t_k;
          row = row_cur;
          const int j = s.k0 + t * kTile + warp * 32 + lane;
          // a key that does not exist; those behind k1 are told by their number alone
          const uint32_t inv = __ballot_sync(0xffffffffu, row < 0 && (MODE == kSelected || j < s.k1));
          if (lane == 0) s_inv[((seen + t) % kKeep) * 4 + warp] = inv;
          if (MODE == kSelected && !PLAIN) s_key[((seen + t) % kKeep) * kTile + warp * 32 + lane] = key_cur;
        } else {
          row = t == t_k - 1 ? row_cur : row_prev;
        }
        uint8_t* dst = ring + slot * L::tile + (c >> 3) * L::half;
        const uint16_t* base = (is_k ? a.c.k : a.c.v) + head + c * 8;
#pragma unroll 4
        for (int u = 0; u < 32 / kPer; ++u) {
          const int r = u * kPer + sub;
          const int64_t off = __shfl_sync(0xffffffffu, row, r);
          const int rr = warp * 32 + r;
          cp_async_16(dst + rr * 128 + (((c & 7) ^ (rr & 7)) << 4), base + (off < 0 ? -head : off), off >= 0);
        }
        cp_async_commit();
        ++cnt;
        if (MODE != kSelected && !is_k && s.k0 + t * kTile + kTile - 1 > s.near) {
          // keys that not every row sees: each lane looks over what it copied
          cp_async_wait_group<0>();
          bool cut = false;
#pragma unroll 4
          for (int u = 0; u < 32 / kPer; ++u) {
            const int rr = warp * 32 + u * kPer + sub;
            if (s.k0 + t * kTile + rr > s.near)
              cut |= cut_infinite<E>(reinterpret_cast<uint4*>(dst + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)));
          }
          if (cut) *s_cut = 1;
          announce(cnt);
        }
        cp_async_wait_group<2>();
        if (cnt - 2 > told) announce(cnt - 2);
      }
      seen += s.n;
    }
    cp_async_wait_group<0>();
    if (cnt > told) announce(cnt);
  } else if (warp < 12) {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    const int x = (warp - 4) >> 2;               // stream
    const int r = ((warp & 3) << 5) + lane;      // row of the stream: its TMEM lane
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + x * 128, tO = tmem + lanes + 256 + x * 128;
    const E tag = E();
    uint32_t n_s = 0, n_o = 0, n_ml = 0;  // phases seen
    int seen = 0;                         // key tiles of the items before
    bool ok = true;
    for (int64_t w = blockIdx.x; ok && w < items; w += gridDim.x) {
      const Span s = span_of<MODE, kRows>(a, s_sum, w);
      if (!s.live) continue;
      const int first_tile = seen;
      seen += s.n;
      const int rr = (PAIR ? x * kTile : 0) + r;  // row of the item
      const bool real = rr < s.it.nrows;
      const int g = s.it.r0 + (real ? rr : 0);
      const int t = s.it.qb + g / a.G, h = s.it.h * a.G + g % a.G;
      int pos = 0x7ffffffe;
      if (real) {
        const int sq = MODE == kShared ? upper_segment<int32_t>(a.qo, a.S, t) : s.it.seq;
        pos = checked_pos(a, t, sq);
      }
      const int64_t row = (int64_t)t * a.Hq + h;
      if (s.n > 0) {
        // this row of Q (in split mode, half of it each), zeros for rows that are not
        constexpr int kC = D / 8 / (PAIR ? 1 : 2);
        const int c0 = PAIR ? 0 : x * kC;
        const uint4* src = reinterpret_cast<const uint4*>(a.q + row * D);
        uint8_t* dst = smem + (PAIR ? x * L::tile : 0) + r * 128;
        uint4 v[kC];
#pragma unroll
        for (int i = 0; i < kC; ++i) v[i] = real ? __ldg(src + c0 + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < kC; ++i) {
          const int c = c0 + i;
          *reinterpret_cast<uint4*>(dst + (c >> 3) * L::half + (((c & 7) ^ (r & 7)) << 4)) = v[i];
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
      }
      float slope = 0.f;
      const bool bias = !PLAIN && a.slopes;
      if (bias) slope = __ldg(a.slopes + h) * kLog2e;
      const float sc = PLAIN ? fabsf(a.scale2) : 1.f;
      const bool flip = PLAIN && a.scale2 < 0.f;
      // contiguous keys: the last one that this row sees
      const int lim = MODE == kSelected ? 0x7fffffff : min(pos, s.k1 - 1);
      const int least = __reduce_min_sync(0xffffffffu, lim);
      const int mine = PAIR ? s.n : (s.n + 1 - x) / 2;
      float ref = -INFINITY, l0 = 0.f, l1 = 0.f;
      for (int i = 0; i < mine; ++i) {
        const int tile = PAIR ? i : 2 * i + x;
        const int base = s.k0 + tile * kTile;
        if (!warp_wait(&s_full[x], n_s & 1, abort, a.status)) { ok = false; break; }
        ++n_s;
        tc_fence_after();
        float v[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(tS + q * 32, v[q]);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 4; ++q) reg_fence32(v[q]);
        if (flip) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < 32; ++j) v[q][j] = -v[q][j];
        }
        if constexpr (!PLAIN) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < 32; ++j) v[q][j] = exponent<false>(v[q][j], a);
          if (bias) {
            if constexpr (MODE == kSelected) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                  const int4 kp = *reinterpret_cast<const int4*>(s_key + ((first_tile + tile) % kKeep) * kTile + q * 32 + j);
                  v[q][j] = fmaf(-slope, (float)(pos - kp.x), v[q][j]);
                  v[q][j + 1] = fmaf(-slope, (float)(pos - kp.y), v[q][j + 1]);
                  v[q][j + 2] = fmaf(-slope, (float)(pos - kp.z), v[q][j + 2]);
                  v[q][j + 3] = fmaf(-slope, (float)(pos - kp.w), v[q][j + 3]);
                }
            } else {
              const float first = (float)(pos - base);
#pragma unroll
              for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int j = 0; j < 32; ++j) v[q][j] = fmaf(-slope, first - (float)(q * 32 + j), v[q][j]);
            }
          }
        }
        if (MODE != kSelected && base + kTile - 1 > least) {
          const int last = lim - base;  // columns up to this one are seen
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (q * 32 + j > last) v[q][j] = -INFINITY;
        }
        {
          const uint4 inv = *reinterpret_cast<const uint4*>(s_inv + ((first_tile + tile) % kKeep) * 4);
          if (inv.x | inv.y | inv.z | inv.w) {
            const uint32_t word[4] = {inv.x, inv.y, inv.z, inv.w};
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (word[q] >> j & 1u) v[q][j] = -INFINITY;
          }
        }
        float top = -INFINITY;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float m0 = v[q][0], m1 = v[q][1];
#pragma unroll
          for (int j = 2; j < 32; j += 2) {
            m0 = fmaxf(m0, v[q][j]);
            m1 = fmaxf(m1, v[q][j + 1]);
          }
          top = fmaxf(top, fmaxf(m0, m1));
        }
        top *= sc;  // sc > 0: -inf stays
        const bool grow = top > ref + kSlack || (ref == -INFINITY && top > -INFINITY);
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? ex2(ref - top) : 1.f;  // 0 while nothing had been seen
          if (grow) ref = top;
          l0 *= f;
          l1 *= f;
          if (i > 0) {
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
              float o[32];
              uint32_t u[32];
              tmem_ld32(tO + q * 32, o);
              tmem_wait_ld();
              reg_fence32(o);
#pragma unroll
              for (int j = 0; j < 32; ++j) u[j] = __float_as_uint(o[j] * f);
              tmem_st32(tO + q * 32, u);
            }
          }
        }
        const float minus = ref == -INFINITY ? 0.f : -ref;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t p[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            float& e0 = v[2 * q + (j >> 4)][(j & 15) * 2];
            float& e1 = v[2 * q + (j >> 4)][(j & 15) * 2 + 1];
            e0 = ex2(fmaf(e0, sc, minus));
            e1 = ex2(fmaf(e1, sc, minus));
            l0 += e0;
            l1 += e1;
            // the weights' one rounding to the cache's type; their sum keeps fp32
            p[j] = pack2(e0, e1, tag);
          }
          tmem_st32(tS + q * 32, p);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
      }
      if (!ok) break;
      float l = l0 + l1;
      if (mine > 0) {
        if (!warp_wait(&o_full[x], n_o & 1, abort, a.status)) break;
        ++n_o;
        tc_fence_after();
      }
      // Weights of the two streams' rows (split), and the end of the row.
      float fa, fb = 0.f, lse2;
      if constexpr (PAIR) {
        fa = l == 0.f ? 0.f : 1.f / l;
        lse2 = l == 0.f ? -INFINITY : ref + lg2(l);
      } else if (s.n == 0) {
        fa = 0.f;  // no keys: nothing to exchange, and the other stream may still read the last item's
        lse2 = -INFINITY;
      } else {
        s_ml[x * kTile + r] = make_float2(ref, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ml_full);
        if (!warp_wait(ml_full, n_ml & 1, abort, a.status)) break;
        ++n_ml;
        const float2 ma = s_ml[r], mb = s_ml[kTile + r];
        const float m = fmaxf(ma.x, mb.x), base = m == -INFINITY ? 0.f : m;
        fa = ma.y == 0.f ? 0.f : ex2(ma.x - base);
        fb = mb.y == 0.f ? 0.f : ex2(mb.x - base);
        l = fmaf(fa, ma.y, fb * mb.y);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        fa *= inv;
        fb *= inv;
        lse2 = l == 0.f ? -INFINITY : base + lg2(l);
        // stream B's O is complete when its thread came to the barrier, A's likewise
        tc_fence_after();
      }
      constexpr int kCols = PAIR ? D : D / 2;  // in split mode A writes the first half of the dims, B the second
      const int d0 = PAIR ? 0 : x * kCols;
      const uint32_t ta = tmem + lanes + 256 + (PAIR ? x * 128 : 0) + d0, tb = tmem + lanes + 384 + d0;
      // values cut out of a tile that this row does see (only rows behind `near` can)
      const int cut0 = max(s.k0, s.near + 1);
      const bool cut = MODE != kSelected && s.n > 0 && real && cut0 <= lim && *s_cut;
      const bool any_a = PAIR ? mine > 0 : s.n > 0, any_b = !PAIR && s.n > 1;
#pragma unroll 1
      for (int q = 0; q < kCols / 32; ++q) {
        float o[32];
        if (any_a) {
          tmem_ld32(ta + q * 32, o);
          tmem_wait_ld();
          reg_fence32(o);
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = any_a && fa != 0.f ? o[j] * fa : 0.f;
        if constexpr (!PAIR) {
          if (any_b) {
            float ob[32];
            tmem_ld32(tb + q * 32, ob);
            tmem_wait_ld();
            reg_fence32(ob);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] += fb != 0.f ? ob[j] * fb : 0.f;
          }
        }
        if (cut) poison<E, 32>(a, s.it.seq, s.it.h, d0 + q * 32, cut0, lim, o);
        if (real) {
          if (a.part_o) {
            float4* d = reinterpret_cast<float4*>(a.part_o + (row * a.nslots + s.it.slot) * D + d0 + q * 32);
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          } else {
            uint4* d = reinterpret_cast<uint4*>(a.out + row * D + d0 + q * 32);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              d[j] = make_uint4(pack2(o[8 * j], o[8 * j + 1], tag), pack2(o[8 * j + 2], o[8 * j + 3], tag),
                                pack2(o[8 * j + 4], o[8 * j + 5], tag), pack2(o[8 * j + 6], o[8 * j + 7], tag));
          }
        }
      }
      if (real && (PAIR || x == 0)) {
        if (a.part_o) a.part_lse[row * a.nslots + s.it.slot] = lse2;
        else if (a.lse) a.lse[row] = lse2 * kLn2;
      }
      tc_fence_before();
    }
  } else {
    // ------------------------------------------------------------ products
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 12) {
      const uint32_t idesc_s = tc_idesc<E>(kTile, false), idesc_o = tc_idesc<E>(D, true);
      const uint32_t q_addr = smem_u32(smem), ring_addr = smem_u32(ring);
      int cnt = 0;
      uint32_t n_q = 0, n_p[2] = {0, 0};
      bool ok = true;
      auto qk = [&](int x, int slot) {
        const uint32_t qa = q_addr + (PAIR ? x * L::tile : 0), ka = ring_addr + slot * L::tile;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * L::half + (kk & 3) * 32;
          umma_bf16(tmem + x * 128, sw128_kmajor_desc(qa + off), sw128_kmajor_desc(ka + off), idesc_s, kk > 0);
        }
      };
      auto pv = [&](int x, int slot, bool acc) {
        const uint32_t va = ring_addr + slot * L::tile;
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          umma_ts(tmem + 256 + x * 128, tmem + x * 128 + kk * 8, sw128_nmajor_desc(va + kk * 2048, L::half), idesc_o,
                  acc || kk > 0);
      };
      for (int64_t w = blockIdx.x; ok && w < items; w += gridDim.x) {
        const Span s = span_of<MODE, kRows>(a, s_sum, w);
        if (s.n == 0) continue;
        if (lane == 0) {
          auto wait_slot = [&](int place) {
            const int i = cnt + place;
            return mbar_wait(&full[i % kSlots], (i / kSlots) & 1, abort, a.status);
          };
          const int n0 = PAIR ? s.n : (s.n + 1) / 2, n1 = PAIR ? s.n : s.n / 2;
          ok = mbar_wait(q_full, n_q & 1, abort, a.status);
          tc_fence_after();
          for (int i = -1; ok && i < n0; ++i) {
            for (int x = 0; ok && x < 2; ++x) {
              const int nx = x ? n1 : n0;
              if (i >= nx) break;
              if (i >= 0) {
                const int t = PAIR ? i : 2 * i + x, place = place_v<PAIR>(t, s.n);
                ok = wait_slot(place) && mbar_wait(&p_full[x], n_p[x]++ & 1, abort, a.status);
                if (!ok) break;
                tc_fence_after();
                pv(x, (cnt + place) % kSlots, i > 0);
                if (!PAIR || x == 1) umma_commit(&empty[(cnt + place) % kSlots]);
              }
              if (i + 1 < nx) {
                const int t = PAIR ? i + 1 : 2 * (i + 1) + x, place = place_k<PAIR>(t);
                if (!(ok = wait_slot(place))) break;
                tc_fence_after();
                qk(x, (cnt + place) % kSlots);
                if (!PAIR || x == 1) umma_commit(&empty[(cnt + place) % kSlots]);
                umma_commit(&s_full[x]);
              } else if (i >= 0) {
                umma_commit(&o_full[x]);
              }
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        ++n_q;
        cnt += 2 * s.n;
      }
      if (lane == 0) {
        // every product must be done before TMEM is given back
        umma_commit(drain);
        mbar_wait(drain, 0, abort, a.status, kDrainCycles, /*drain=*/true);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <typename E, int D, int MODE, bool PAIR, bool PLAIN>
int launch_tc_one(const AttendArgs& a, int64_t bound, cudaStream_t st) {
  using L = Tc<D, PAIR>;
  auto kern = attend_tc_kernel<E, D, MODE, PAIR, PLAIN>;
  int rc = set_smem_limit((const void*)kern, L::bytes);
  if (rc) return rc;
  // The roles' register counts add up to what a block of 128-register threads
  // is launched with; a build that used fewer would wait for registers for good.
  static const int regs = [&] {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, kern) == cudaSuccess ? fa.numRegs : 0;
  }();
  if (regs != 128) {
    set_error("attend_tc: built with %d registers a thread, needs 128", regs);
    return MISA_ERR_CUDA;
  }
  const int64_t sms = num_sms();
  const unsigned grid = (unsigned)(bound < 1 ? 1 : bound < sms ? bound : sms);
  static const char* const names[] = {"attend_tc", "attend_tc_shared", "attend_tc_selected"};
  ProfScope ps(names[MODE], st);
  return cuda_fail(launch_pdl(kern, dim3(grid), dim3(kTcThreads), L::bytes, st, a), "attend_tc_kernel");
}

template <typename E, int D, int MODE, bool PAIR>
int launch_tc_kind(const AttendArgs& a, int64_t bound, cudaStream_t st) {
  // a scale of 0 times a masked -inf: the other form scales before it masks
  return a.cap2 > 0.f || a.slopes || a.scale2 == 0.f ? launch_tc_one<E, D, MODE, PAIR, false>(a, bound, st)
                                  : launch_tc_one<E, D, MODE, PAIR, true>(a, bound, st);
}

template <int MODE, bool PAIR>
int launch_tc_type(const AttendArgs& a, int dtype, int D, int64_t bound, cudaStream_t st) {
  if (dtype == MISA_BF16)
    return D == 128 ? launch_tc_kind<__nv_bfloat16, 128, MODE, PAIR>(a, bound, st)
                    : launch_tc_kind<__nv_bfloat16, 64, MODE, PAIR>(a, bound, st);
  return D == 128 ? launch_tc_kind<__half, 128, MODE, PAIR>(a, bound, st)
                  : launch_tc_kind<__half, 64, MODE, PAIR>(a, bound, st);
}

}  // namespace

// rows: 128 (split) or 256 (pair) rows of an item.
int launch_attend_tc(const AttendArgs& a, int mode, int rows, int dtype, int D, int64_t bound, cudaStream_t st) {
  if (mode == kSelected) return launch_tc_type<kSelected, false>(a, dtype, D, bound, st);
  if (mode == kShared)
    return rows == 128 ? launch_tc_type<kShared, false>(a, dtype, D, bound, st)
                       : launch_tc_type<kShared, true>(a, dtype, D, bound, st);
  return rows == 128 ? launch_tc_type<kOwn, false>(a, dtype, D, bound, st)
                     : launch_tc_type<kOwn, true>(a, dtype, D, bound, st);
}

}  // namespace misa
