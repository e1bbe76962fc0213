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
// Warps 0-3 and 4-7 are the softmax of A and B.  Warp 8 issues the products
// (one thread).  Warp 9 finds where the rows of each tile lie; warps 10, 11
// (keys) and 12, 13 (values) fetch them into a ring of 128-row tiles, 128-byte
// swizzled: a tile of whole pages by TMA boxes, any other, and a selection, by
// TMA gathers of four rows (a row that does not exist is out of the map's bounds
// and comes as zeros).  A thread issues a gather in about 35 cycles, so two share
// a tile (gathers by one thread an SM read 3.2 TB/s from L2, by four 12.6).
// Warp 14 looks over value tiles that only some rows see (cut_infinite).  Where a
// block takes several items, the fetching warps run ahead into the next one.
//
// Bound by the chain of one tile (its S, two passes of softmax, P, the product:
// about 4000 cycles, of which the other stream hides half): 2 x 1000 queries of
// 32 heads behind 16384 tokens, with a bias, take 503 us (776 TF/s; tensor and
// special-function pipes 42% busy), 3000 selections of 2048 for 64 heads 523 us.
#include <algorithm>
#include <type_traits>

#include "attend.cuh"

namespace misa {
namespace {

constexpr int kTcThreads = 512;
constexpr int kTile = 128;          // keys of a tile, rows of a stream
constexpr int kAbove = 8;           // log2 of how far a row's maximum may outgrow its reference
constexpr int kPrep = 2;            // tiles whose rows have been found and not been fetched
constexpr int kKeep = 8;            // tiles whose key masks are kept

template <int D, bool PAIR>
struct Tc {
  static constexpr int lead = PAIR ? 1 : 2;                // key tiles fetched before their values
  static constexpr int halves = D / 64;
  static constexpr int half = kTile * 128;                 // 64 dims of a tile
  static constexpr int tile = half * halves;
  static constexpr int q_tiles = PAIR ? 2 : 1;
  static constexpr int slots = D == 128 ? 5 : 10;
  static constexpr int off_ring = q_tiles * tile;
  static constexpr int off_far = off_ring + slots * tile;  // distances, selected mode with a bias
  static constexpr int off_inv = off_far + (PAIR ? 0 : kKeep * kTile * 4);
  static constexpr int off_ml = off_inv + kKeep * 16;
  static constexpr int off_rows = off_ml + (PAIR ? 0 : 2 * kTile * 8);
  static constexpr int off_bar = off_rows + kPrep * kTile * 4;
  static constexpr int bars = 2 * slots + 13 + 2 * kPrep;
  static constexpr int off_sum = off_bar + bars * 8;
  static constexpr int bytes = off_sum + 16 + (kScan + 1 + kScan / 32) * 4 + 1024;
  static_assert(bytes <= 227 * 1024, "shared memory of a block");
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

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32],"
      " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"f"(r[0]),
      "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]), "f"(r[9]),
      "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15]), "f"(r[16]), "f"(r[17]),
      "f"(r[18]), "f"(r[19]), "f"(r[20]), "f"(r[21]), "f"(r[22]), "f"(r[23]), "f"(r[24]), "f"(r[25]),
      "f"(r[26]), "f"(r[27]), "f"(r[28]), "f"(r[29]), "f"(r[30]), "f"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16],"
      " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// What every role works out for itself about an item.
struct Span {
  Item it;
  int k0, k1, n;  // keys, and tiles of them
  int cut;        // tiles before this one hold keys which not all rows see
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
    s.k0 = s.it.k0 & ~(a.box_align - 1);  // tiles start where a box can; keys before it.k0 are masked
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
  s.n = s.live && s.k1 > s.it.k0 ? (s.k1 - s.k0 + kTile - 1) / kTile : 0;
  s.cut = 0;
  if (MODE != kSelected && s.near < s.k1 - 1) s.cut = s.n - (s.near < s.k0 ? 0 : min(s.n, (s.near + 1 - s.k0) / kTile));
  return s;
}

// First key of tile t.  Contiguous keys come last first: with a bias that falls
// with the distance the row's maximum is then near its end at once, and no
// later tile makes it grow (a rescaling of O costs a tile half its softmax).
template <int MODE>
__device__ __forceinline__ int tile_start(const Span& s, int t) {
  return s.k0 + (MODE == kSelected ? t : s.n - 1 - t) * kTile;
}

// Order of the ring: `lead` key tiles, then value tile t and key tile t + lead
// in turn.  Place of value tile t among an item's 2 n tiles:
template <bool PAIR>
__device__ __forceinline__ int place_v(int t, int n) {
  constexpr int lead = PAIR ? 1 : 2;
  return t + min(t + lead, n);
}

template <bool PAIR>
__device__ __forceinline__ int place_k(int t) {
  constexpr int lead = PAIR ? 1 : 2;
  return t < lead ? t : 2 * t - lead + 1;
}

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// A load that stays where it is written, ahead of copies that it does not depend on.
__device__ __forceinline__ int load_early(const int32_t* p) {
  int r;
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(r) : "l"(p));
  return r;
}

// Four rows of 64 elements, from element x of each on.
__device__ __forceinline__ void tma_gather4(const CUtensorMap* map, uint64_t* bar, void* dst, int x, const int4& r) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w)
      : "memory");
}

// A box of rows from place `off` of a page on, 64 elements of each from element x on.
__device__ __forceinline__ void tma_box(const CUtensorMap* map, uint64_t* bar, void* dst, int x, int off, int head,
                                        int page) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(off), "r"(head), "r"(page)
      : "memory");
}

// rows: the cache as [map_rows, D], for gathers of any rows; boxes: as
// [pages, heads, page, D], for runs of `box` rows of one page.
struct TcMaps {
  CUtensorMap rows[2], boxes[2];  // keys, values
};

template <typename E, int D, int MODE, bool PAIR, int KIND>
__global__ void __launch_bounds__(kTcThreads, 1)
attend_tc_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ TcMaps maps) {
  pdl_wait_then_release();
  using L = Tc<D, PAIR>;
  constexpr int kRows = kTile * L::q_tiles;
  constexpr int kSlots = L::slots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + L::off_ring;
  float* s_far = reinterpret_cast<float*>(smem + L::off_far);
  uint32_t* s_inv = reinterpret_cast<uint32_t*>(smem + L::off_inv);
  float2* s_ml = reinterpret_cast<float2*>(smem + L::off_ml);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::off_bar);
  uint64_t* empty = full + kSlots;
  uint64_t* s_full = empty + kSlots;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 4;
  uint64_t* q_full = o_full + 2;
  uint64_t* ml_full = q_full + 1;
  uint64_t* drain = ml_full + 1;
  uint64_t* cut_ask = drain + 1;
  uint64_t* cut_done = cut_ask + 1;
  uint64_t* prep_full = cut_done + 1;
  uint64_t* prep_empty = prep_full + kPrep;
  int4* s_rows = reinterpret_cast<int4*>(smem + L::off_rows);  // a tile's rows, or its boxes' places and pages
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::off_sum);
  int* abort = reinterpret_cast<int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  volatile int* s_cut = abort + 1;  // something was cut out of a value tile of this block
  volatile int* s_boxed = abort + 2;  // bit i: entry i of s_rows holds boxes
  int* s_sum = abort + 3;
  int total;
  if (MODE == kShared && blockIdx.x == 0) check_shared(a);
  if constexpr (MODE == kSelected) {
    total = a.T * ((a.G + kRows - 1) / kRows) * a.nch_max;
  } else {
    total = count_items<MODE>(a, kRows, s_sum);
  }
  const int64_t items = (int64_t)total * a.Hkv;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&full[i], 2);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[2 * i], 4);
      mbar_init(&p_full[2 * i + 1], 4);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(q_full, 8);
    mbar_init(ml_full, 8);
    mbar_init(drain, 1);
    mbar_init(cut_ask, 1);
    mbar_init(cut_done, 1);
    for (int i = 0; i < kPrep; ++i) {
      mbar_init(&prep_full[i], 1);
      mbar_init(&prep_empty[i], 4);
    }
    *s_boxed = 0;
    *abort = 0;
    *s_cut = 0;
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    const int x = warp >> 2;                     // stream
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
      const bool idle = rr - lane >= s.it.nrows;  // no row of this warp is
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
      const bool bias = KIND == kBiased || (KIND == kCapped && a.slopes);
      if (a.slopes && bias) slope = __ldg(a.slopes + h) * kLog2e;
      const float sc = KIND == kScaled ? a.scale2 : 1.f;
      // contiguous keys: the last one that this row sees
      const int lim = MODE == kSelected ? 0x7fffffff : min(pos, s.k1 - 1);
      const int least = __reduce_min_sync(0xffffffffu, lim);
      const int mine = PAIR ? s.n : (s.n + 1 - x) / 2;
      float ref = -INFINITY;
      uint64_t l01 = pair(0.f, 0.f);  // the row's sum: even and odd keys
      const uint64_t sc2 = pair(sc, sc);
      for (int i = 0; i < mine; ++i) {
        const int tile = PAIR ? i : 2 * i + x;
        const int base = tile_start<MODE>(s, tile);
        if (!warp_wait(&s_full[x], n_s & 1, abort, a.status)) { ok = false; break; }
        ++n_s;
        if (idle) {  // what these rows of S hold as P reaches no other row
          if (lane < 2) mbar_arrive(&p_full[2 * x + lane]);
          continue;
        }
        tc_fence_after();
        float v[2][32];
        tmem_ld32(tS, v[0]);
        const int last = lim - base;  // contiguous keys: columns up to this one are seen
        const int keep = (first_tile + tile) % kKeep;
        const uint4 inv = *reinterpret_cast<const uint4*>(s_inv + keep * 4);
        const bool masked = (MODE != kSelected && base + kTile - 1 > least) || (inv.x | inv.y | inv.z | inv.w);
        // What is done to the products, in place and back to S where it is not nothing, and the
        // maximum; 32 columns at a time, the next ones' load under way.
        float top = -INFINITY;
        auto piece = [&](int q, float (&u)[32]) {
          auto mask = [&](float value) {  // what this row does not see gets `value`
            if (!masked) return;
            const uint32_t word = q == 0 ? inv.x : q == 1 ? inv.y : q == 2 ? inv.z : inv.w;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if ((MODE != kSelected && j > last - q * 32) || (word >> j & 1u)) u[j] = value;
          };
          if constexpr (KIND == kCapped) {
            mask(0.f);
            float most = 0.f;
#pragma unroll
            for (int j = 0; j < 32; j += 2) most = max3_abs(most, u[j], u[j + 1]);
            if (__all_sync(0xffffffffu, most < a.series_max)) {
#pragma unroll
              for (int j = 0; j < 32; j += 2) cap_series(u[j], u[j + 1], a);
            } else {
#pragma unroll
              for (int j = 0; j < 32; j += 2) cap_any(u[j], u[j + 1], a);
            }
          }
          if (bias) {
            const uint64_t mul = KIND == kCapped ? pair(1.f, 1.f) : pair(a.scale2, a.scale2);
            const float* far = s_far + keep * kTile + q * 32;
            const float first = -slope * (float)(pos - base - q * 32);
            const uint64_t step = pair(2.f * slope, 2.f * slope), minus = pair(-slope, -slope);
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              // slope times the distance: for contiguous keys three steps from an exact start
              uint64_t b[4];
              if constexpr (MODE == kSelected) {
                const float4 d = *reinterpret_cast<const float4*>(far + j);
                const float4 e = *reinterpret_cast<const float4*>(far + j + 4);
                b[0] = mul2(minus, pair(d.x, d.y)), b[1] = mul2(minus, pair(d.z, d.w));
                b[2] = mul2(minus, pair(e.x, e.y)), b[3] = mul2(minus, pair(e.z, e.w));
              } else {
                b[0] = pair(fmaf(slope, (float)j, first), fmaf(slope, (float)(j + 1), first));
#pragma unroll
                for (int i = 1; i < 4; ++i) b[i] = add2(b[i - 1], step);
              }
#pragma unroll
              for (int i = 0; i < 4; ++i)
                unpair(fma2(pair(u[j + 2 * i], u[j + 2 * i + 1]), mul, b[i]), u[j + 2 * i], u[j + 2 * i + 1]);
            }
          }
          mask(-INFINITY);
          float t0 = u[0], t1 = u[1];
#pragma unroll
          for (int j = 2; j < 30; j += 4) {
            t0 = max3(t0, u[j], u[j + 1]);
            t1 = max3(t1, u[j + 2], u[j + 3]);
          }
          top = max3(top, max3(t0, u[30], u[31]), t1);
          if (KIND != kScaled || masked) tmem_st32(tS + q * 32, u);
        };
#pragma unroll 1
        for (int q = 0; q < 4; q += 2) {
          tmem_wait_ld();
          reg_fence32(v[0]);
          tmem_ld32(tS + q * 32 + 32, v[1]);
          piece(q, v[0]);
          tmem_wait_ld();
          reg_fence32(v[1]);
          if (q == 0) tmem_ld32(tS + 64, v[0]);
          piece(q + 1, v[1]);
        }
        if (KIND != kScaled || masked) tmem_wait_st();
        top *= sc;  // sc > 0: -inf stays
        // an infinite or undefined exponent makes the row's results undefined
        if (!(top < INFINITY)) top = __int_as_float(0x7fffffff);
        const bool grow = top > ref + kAbove || (ref == -INFINITY && top > -INFINITY) || top != top;
        if (__any_sync(0xffffffffu, grow)) {
          const float f = grow ? ex2(reference<E, kAbove>(ref) - reference<E, kAbove>(top)) : 1.f;  // 0 while nothing had been seen
          if (grow) ref = top;
          l01 = mul2(l01, pair(f, f));
          if (i > 0) {
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
              float o[32];
              tmem_ld32(tO + q * 32, o);
              tmem_wait_ld();
              reg_fence32(o);
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] *= f;
              tmem_st32(tO + q * 32, o);
            }
          }
        }
        const float minus = ref == -INFINITY ? 0.f : -reference<E, kAbove>(ref);
        const uint64_t minus2 = pair(minus, minus);
        auto weigh = [&](int q, const float (&u)[32]) {
          uint32_t p[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            uint64_t e = pair(u[2 * j], u[2 * j + 1]);
            float e0, e1;
            e = KIND == kScaled ? fma2(e, sc2, minus2) : add2(e, minus2);
            unpair(e, e0, e1);
            e0 = ex2(e0);
            e1 = ex2(e1);
            e = pair(e0, e1);
            l01 = add2(l01, e);
            // the weights' one rounding to the cache's type; their sum keeps fp32
            p[j] = pack2(e0, e1, tag);
          }
          tmem_st16(tS + q * 16, p);
        };
        tmem_ld32(tS, v[0]);
#pragma unroll 1
        for (int q = 0; q < 4; q += 2) {
          tmem_wait_ld();
          reg_fence32(v[0]);
          tmem_ld32(tS + q * 32 + 32, v[1]);
          weigh(q, v[0]);
          tmem_wait_ld();
          reg_fence32(v[1]);
          if (q == 0) tmem_ld32(tS + 64, v[0]);
          weigh(q + 1, v[1]);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * x + (q >> 1)]);  // half of the keys
        }
      }
      if (!ok) break;
      ref = reference<E, kAbove>(ref);
      float l0, l1;
      unpair(l01, l0, l1);
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
        lse2 = l == 0.f ? -INFINITY : log_sum<E, kAbove>(ref, l);
      } else if (s.n == 0) {
        fa = 0.f;  // no keys: nothing to exchange, and the other stream may still read the last item's
        lse2 = -INFINITY;
      } else {
        // a stream without tiles leaves nothing: it has not waited for a product of this item, so the
        // other may still be reading what the last item's rows left in its place
        if (mine > 0) s_ml[x * kTile + r] = make_float2(ref, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ml_full);
        if (!warp_wait(ml_full, n_ml & 1, abort, a.status)) break;
        ++n_ml;
        const float2 ma = s_ml[r], mb = s.n > 1 ? s_ml[kTile + r] : make_float2(-INFINITY, 0.f);
        const float m = fmaxf(ma.x, mb.x), base = m == -INFINITY ? 0.f : m;
        fa = ma.y == 0.f ? 0.f : ex2(ma.x - base);
        fb = mb.y == 0.f ? 0.f : ex2(mb.x - base);
        l = fmaf(fa, ma.y, fb * mb.y);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        fa *= inv;
        fb *= inv;
        lse2 = l == 0.f ? -INFINITY : log_sum<E, kAbove>(base, l);
        // stream B's O is complete when its thread came to the barrier, A's likewise
        tc_fence_after();
      }
      constexpr int kCols = PAIR ? D : D / 2;  // in split mode A writes the first half of the dims, B the second
      const int d0 = PAIR ? 0 : x * kCols;
      const uint32_t ta = tmem + lanes + 256 + (PAIR ? x * 128 : 0) + d0, tb = tmem + lanes + 384 + d0;
      // values cut out of a tile that this row does see (only rows behind `near` can)
      const int cut0 = max(s.it.k0, s.near + 1);
      const bool cut = MODE != kSelected && s.n > 0 && real && cut0 <= lim && *s_cut;
      const bool any_a = PAIR ? mine > 0 : s.n > 0, any_b = !PAIR && s.n > 1;
#pragma unroll 1
      for (int q = 0; q < kCols / 32 && !idle; ++q) {
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
    if (warp == 9) {
      // ---------------------------------------------------------- finding rows
      // lane l finds keys 4 l .. 4 l + 3 of a tile
      int seen = 0;  // key tiles of the items before
      bool ok = true;
      for (int64_t w = blockIdx.x; ok && w < items; w += gridDim.x) {
        const Span s = span_of<MODE, kRows>(a, s_sum, w);
        if (s.n == 0) continue;
        const int head = s.it.h * a.head_rows;
        const int64_t first_row = a.c.table ? 0 : __ldg(a.c.ko + s.it.seq);  // packed
        const int pos = MODE == kSelected ? __ldg(a.q_pos + s.it.qb) : 0;
        const int32_t* list = a.idx + (int64_t)s.it.qb * a.k;
        const int32_t* table = a.c.table + s.it.seq * a.c.table_stride;
        auto keys_of = [&](int t, int (&key)[4]) {
          const int j = tile_start<MODE>(s, t) + lane * 4;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            key[i] = -1;
            if (t < s.n && j + i >= s.it.k0 && j + i < s.k1) key[i] = MODE == kSelected ? load_early(list + j + i) : j + i;
          }
        };
        // Page and place in it of each key, and the page table's entry, read whether it is needed
        // or not: four loads in flight.  (One test of the page size: divisions cost more than the copies.)
        auto pages_of = [&](const int (&key)[4], int (&page)[4], int (&off)[4]) {
          if (!a.c.table) return;
          if (a.c.page_shift >= 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              page[i] = max(key[i], 0) >> a.c.page_shift;
              off[i] = max(key[i], 0) & (a.c.page_size - 1);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              page[i] = max(key[i], 0) / a.c.page_size;
              off[i] = max(key[i], 0) - page[i] * a.c.page_size;
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) page[i] = page[i] < a.c.pages_per_seq ? load_early(table + page[i]) : -1;
        };
        // a tile's keys and pages, and the next one's keys
        int key[4], page[4] = {0, 0, 0, 0}, off[4] = {0, 0, 0, 0}, next[4];
        keys_of(0, key);
        pages_of(key, page, off);
        keys_of(1, next);
        for (int t = 0; t < s.n; ++t) {
          const int start = tile_start<MODE>(s, t);
          int row[4];
          uint32_t bad = 0, none = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool ahead = MODE == kSelected && key[i] > pos;
            const int r = cache_unit(a, first_row, max(key[i], 0), page[i], off[i]);
            const bool there = key[i] >= 0 && !ahead && r >= 0;
            if (key[i] >= 0 && !there) bad |= ahead ? MISA_STATUS_BAD_INPUT : MISA_STATUS_BOUNDS;
            row[i] = there ? head + r : a.map_rows;  // out of the map's bounds: zeros
            // keys that do not exist; those behind k1 of contiguous ones are told by their number alone
            if (!there && (MODE == kSelected || start + lane * 4 + i < s.k1)) none |= 1u << i;
          }
          if (bad) set_status(a.status, bad);
          uint32_t word = 0;
          const bool whole = !__any_sync(0xffffffffu, none != 0);
          if (!whole) {
            word = none << (4 * (lane & 7));
            word |= __shfl_xor_sync(0xffffffffu, word, 1);
            word |= __shfl_xor_sync(0xffffffffu, word, 2);
            word |= __shfl_xor_sync(0xffffffffu, word, 4);
          }
          const bool boxed = MODE != kSelected && a.box > 0 && whole && start + kTile <= s.k1;
          const float4 far = make_float4(pos - key[0], pos - key[1], pos - key[2], pos - key[3]);
          const int2 place = a.c.table ? make_int2(off[0], page[0]) : make_int2((int)first_row + key[0], 0);
          // the loads of the tiles to come run while this one waits
#pragma unroll
          for (int i = 0; i < 4; ++i) key[i] = next[i];
          pages_of(key, page, off);
          keys_of(t + 2, next);
          const int entry = (seen + t) % kPrep, keep = (seen + t) % kKeep;
          ok = warp_wait(&prep_empty[entry], (((seen + t) / kPrep) & 1) ^ 1, abort, a.status);
          if (!ok) break;
          if ((lane & 7) == 0) s_inv[keep * 4 + (lane >> 3)] = word;
          if (MODE == kSelected && KIND != kScaled) *reinterpret_cast<float4*>(s_far + keep * kTile + lane * 4) = far;
          int4* rows = s_rows + entry * 32;
          if (!boxed) rows[lane] = make_int4(row[0], row[1], row[2], row[3]);
          else if (lane * 4 % a.box == 0) reinterpret_cast<int2*>(rows)[lane * 4 / a.box] = place;
          if (lane == 0) *s_boxed = (*s_boxed & ~(1 << entry)) | (boxed ? 1 << entry : 0);
          __syncwarp();
          if (lane == 0) mbar_arrive(&prep_full[entry]);
        }
        seen += s.n;
      }
    } else if (warp >= 10 && warp < 14) {
      // ---------------------------------------------------------- fetching: keys 10, 11, values 12, 13
      // each warp half of a tile's rows; elect, not lane == 0 (see below)
      const bool is_v = warp >= 12;
      const int half = warp & 1;
      int cnt = 0;   // places of the ring taken by the items before
      int seen = 0;  // tiles of the items before
      int last = -1;       // the last place filled; bit i of mine: place last - i was filled by this warp
      uint32_t mine = 0;
      bool ok = true;
      for (int64_t w = blockIdx.x; ok && w < items; w += gridDim.x) {
        const Span s = span_of<MODE, kRows>(a, s_sum, w);
        if (elect_one()) {
          for (int t = 0; t < s.n; ++t) {
            const int place = cnt + (is_v ? place_v<PAIR>(t, s.n) : place_k<PAIR>(t));
            const int slot = place % kSlots, entry = (seen + t) % kPrep;
            ok = mbar_wait(&prep_full[entry], ((seen + t) / kPrep) & 1, abort, a.status) &&
                 mbar_wait(&empty[slot], ((place / kSlots) & 1) ^ 1, abort, a.status);
            if (!ok) break;
            uint64_t* bar = &full[slot];
            mbar_arrive_expect_tx(bar, L::tile / 2);
            mine = mine << (place - last) | 1u;
            last = place;
            uint8_t* dst = ring + slot * L::tile + half * (L::half / 2);
            if (MODE != kSelected && (*s_boxed >> entry & 1)) {
              const int n = kTile / 2 / a.box;
              const int2* at = reinterpret_cast<const int2*>(s_rows + entry * 32) + half * n;
              for (int b = 0; b < n; ++b) {
                const int2 x = at[b];
#pragma unroll
                for (int u = 0; u < L::halves; ++u)
                  tma_box(is_v ? &maps.boxes[1] : &maps.boxes[0], bar, dst + u * L::half + b * a.box * 128, u * 64, x.x,
                          s.it.h, x.y);
              }
            } else {
              const int4* rows = s_rows + entry * 32 + half * 16;
#pragma unroll 8
              for (int g = 0; g < 16; ++g) {
                const int4 r = rows[g];
#pragma unroll
                for (int u = 0; u < L::halves; ++u)
                  tma_gather4(is_v ? &maps.rows[1] : &maps.rows[0], bar, dst + u * L::half + g * 512, u * 64, r);
              }
            }
            mbar_arrive(&prep_empty[entry]);
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        seen += s.n;
        cnt += 2 * s.n;
      }
      // after giving up: this warp's copies still in flight land before the block ends
      if (!ok && elect_one())
        for (int i = 0; i < kSlots && i <= last; ++i)
          if (mine >> i & 1u)
            mbar_wait(&full[(last - i) % kSlots], ((last - i) / kSlots) & 1, abort, a.status, kDrainCycles, /*drain=*/true);
    } else if (warp == 8) {
      // ---------------------------------------------------------- products
      const uint32_t q_addr = smem_u32(smem), ring_addr = smem_u32(ring);
      constexpr uint32_t idesc_s = tc_idesc<E>(kTile, false), idesc_o = tc_idesc<E>(D, true);
      int slot = 0, turn = 0;
      uint32_t n_q = 0, n_p0 = 0, n_p1 = 0, n_cut = 0;
      bool ok = true;
      auto qk = [&](int x, int slot) {
        const uint64_t qd = sw128_kmajor_desc(q_addr + (PAIR ? x * L::tile : 0));
        const uint64_t kd = sw128_kmajor_desc(ring_addr + slot * L::tile);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * L::half + (kk & 3) * 32) >> 4;
          umma_bf16(tmem + x * 128, qd + off, kd + off, idesc_s, kk > 0);
        }
      };
      auto pv = [&](int x, int slot, bool acc, int half) {
        const uint64_t vd = sw128_nmajor_desc(ring_addr + slot * L::tile, L::half);
#pragma unroll
        for (int kk = half * kTile / 32; kk < (half + 1) * kTile / 32; ++kk)
          umma_ts(tmem + 256 + x * 128, tmem + x * 128 + kk * 8, vd + ((kk * 2048) >> 4), idesc_o, acc || kk > 0);
      };
      for (int64_t w = blockIdx.x; ok && w < items; w += gridDim.x) {
        const Span s = span_of<MODE, kRows>(a, s_sum, w);
        if (s.n == 0) continue;
        // elect, not lane == 0: the compiler then knows that one thread issues, and an
        // instruction costs half the issue slots, which the softmax warps compete for
        if (elect_one()) {
          // the next tile of the ring, once it has arrived; -1: given up
          auto take = [&]() -> int {
            const int i = slot;
            if (!mbar_wait(&full[i], turn, abort, a.status)) return -1;
            if (++slot == kSlots) slot = 0, turn ^= 1;
            tc_fence_after();
            return i;
          };
          // stream x's tile of keys
          auto first_product = [&](int x, int k) {
            qk(x, k);
            umma_commit(&s_full[x]);
          };
          auto second_product = [&](int x, int v, bool acc) {
            const uint32_t phase = (x ? n_p1++ : n_p0++) & 1;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              if (!mbar_wait(&p_full[2 * x + half], phase, abort, a.status)) return false;
              tc_fence_after();
              pv(x, v, acc, half);
            }
            return true;
          };
          // value tile t, looked over if not all rows see it
          auto take_v = [&](int t) -> int {
            const int v = take();
            if (v < 0 || t >= s.cut) return v;
            mbar_arrive(cut_ask);
            if (!mbar_wait(cut_done, n_cut++ & 1, abort, a.status)) return -1;
            return v;
          };
          ok = mbar_wait(q_full, n_q & 1, abort, a.status);
          tc_fence_after();
          for (int t = 0; ok && t < min(L::lead, s.n); ++t) {
            const int k = take();
            if (!(ok = k >= 0)) break;
            first_product(t & 1, k);
            if (PAIR) first_product(1, k);
            umma_commit(&empty[k]);
          }
          for (int t = 0; ok && t < s.n; ++t) {
            const int x = PAIR ? 0 : t & 1;
            const bool more = t + L::lead < s.n;
            const int v = take_v(t);
            if (!(ok = v >= 0 && second_product(x, v, t >= L::lead))) break;
            int k = 0;
            if (more) {
              k = take();
              if (!(ok = k >= 0)) break;
              first_product(x, k);
            } else {
              umma_commit(&o_full[x]);
            }
            if (PAIR) {
              if (!(ok = second_product(1, v, t >= L::lead))) break;
              umma_commit(&empty[v]);
              if (more) first_product(1, k);
              else umma_commit(&o_full[1]);
            } else {
              umma_commit(&empty[v]);
            }
            if (more) umma_commit(&empty[k]);
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        ++n_q;
      }
      if (elect_one()) {  // the same thread as above
        // every product must be done before TMEM is given back
        umma_commit(drain);
        mbar_wait(drain, 0, abort, a.status, kDrainCycles, /*drain=*/true);
      }
    } else if (warp == 14 && MODE != kSelected) {
      // ---------------------------------------------------------- looking over values
      int cnt = 0;
      uint32_t n_cut = 0;
      bool ok = true;
      for (int64_t w = blockIdx.x; ok && w < items; w += gridDim.x) {
        const Span s = span_of<MODE, kRows>(a, s_sum, w);
        for (int t = 0; ok && t < s.cut; ++t) {
          const int i = cnt + place_v<PAIR>(t, s.n);
          ok = warp_wait(cut_ask, n_cut++ & 1, abort, a.status) &&
               warp_wait(&full[i % kSlots], (i / kSlots) & 1, abort, a.status);
          if (!ok) break;
          uint8_t* tile = ring + (i % kSlots) * L::tile;
          const int from = s.near + 1 - tile_start<MODE>(s, t);  // rows of the tile from here on
          bool cut = false;
          for (int r = max(from, 0); r < kTile; ++r) {
            // a row's chunks lie in its 128 bytes of each half, in some order
            if (lane < D / 8) cut |= cut_infinite<E>(reinterpret_cast<uint4*>(tile + (lane >> 3) * L::half + r * 128) + (lane & 7));
          }
          if (cut) *s_cut = 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(cut_done);
        }
        cnt += 2 * s.n;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <typename E, int D, int MODE, bool PAIR, int KIND>
int launch_tc_one(const AttendArgs& a, const TcMaps& maps, int64_t bound, cudaStream_t st) {
  using L = Tc<D, PAIR>;
  auto kern = attend_tc_kernel<E, D, MODE, PAIR, KIND>;
  int rc = set_smem_limit((const void*)kern, L::bytes);
  if (rc) return rc;
  // A selection's items are short and alike: one block an SM walks them.  Others are long, and their
  // lengths differ: a block each, which the hardware hands out (2 x 1000 queries: 563 -> 514 us).
  const int64_t most = MODE == kSelected ? num_sms() : 0x7fffffff;
  const unsigned grid = (unsigned)std::max<int64_t>(1, std::min(bound, most));
  static const char* const names[] = {"attend_tc", "attend_tc_shared", "attend_tc_selected"};
  ProfScope ps(names[MODE], st);
  return cuda_fail(launch_pdl(kern, dim3(grid), dim3(kTcThreads), L::bytes, st, a, maps),
                   "attend_tc_kernel");
}

template <typename E, int D, int MODE, bool PAIR>
int launch_tc_kind(const AttendArgs& a, const TcMaps& m, int64_t bound, cudaStream_t st) {
  // the scaled form takes the maximum before it scales: a scale that is not positive goes to the biased one
  return a.cap2 > 0.f                         ? launch_tc_one<E, D, MODE, PAIR, kCapped>(a, m, bound, st)
         : a.slopes || !(a.scale2 > 0.f) ? launch_tc_one<E, D, MODE, PAIR, kBiased>(a, m, bound, st)
                                              : launch_tc_one<E, D, MODE, PAIR, kScaled>(a, m, bound, st);
}

template <int MODE, bool PAIR>
int launch_tc_type(const AttendArgs& a, const TcMaps& m, int dtype, int D, int64_t bound, cudaStream_t st) {
  if (dtype == MISA_BF16)
    return D == 128 ? launch_tc_kind<__nv_bfloat16, 128, MODE, PAIR>(a, m, bound, st)
                    : launch_tc_kind<__nv_bfloat16, 64, MODE, PAIR>(a, m, bound, st);
  return D == 128 ? launch_tc_kind<__half, 128, MODE, PAIR>(a, m, bound, st)
                  : launch_tc_kind<__half, 64, MODE, PAIR>(a, m, bound, st);
}

}  // namespace

// rows: 128 (split) or 256 (pair) rows of an item.
int launch_attend_tc(const AttendArgs& a, int mode, int rows, int dtype, int D, int64_t bound, cudaStream_t st) {
  TcMaps m;
  for (int i = 0; i < 2; ++i) {
    const void* base = i ? a.c.v : a.c.k;
    int rc = make_rows_map(&m.rows[i], base, a.map_rows, D, a.unit, dtype == MISA_FP16);
    if (!rc && a.box) rc = make_box_map(&m.boxes[i], base, a.c, a.Hkv, D, a.box, dtype == MISA_FP16);
    if (rc) return rc;
  }
  if (mode == kSelected) return launch_tc_type<kSelected, false>(a, m, dtype, D, bound, st);
  if (mode == kShared)
    return rows == 128 ? launch_tc_type<kShared, false>(a, m, dtype, D, bound, st)
                       : launch_tc_type<kShared, true>(a, m, dtype, D, bound, st);
  return rows == 128 ? launch_tc_type<kOwn, false>(a, m, dtype, D, bound, st)
                     : launch_tc_type<kOwn, true>(a, m, dtype, D, bound, st);
}

}  // namespace misa
