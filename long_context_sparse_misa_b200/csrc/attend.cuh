// What the attention kernels share: their arguments, the division of a batch
// into work items, the change of a product into a softmax exponent, and how
// partial results are kept.
#pragma once

#include <type_traits>

#include "cache.cuh"

namespace misa {

// Which keys a launch covers.
enum AttendMode { kOwn = 0, kShared = 1, kSelected = 2 };

struct AttendArgs {
  CacheView c;
  const uint16_t* q;   // [T, Hq, D]
  uint16_t* out;       // [T, Hq, D]
  float* lse;          // [T, Hq] or nullptr
  const int32_t* qo;   // [S + 1]
  const int32_t* q_pos;
  const int32_t* idx;  // [T, k], selected mode
  const int32_t* so;   // [ng + 1] shared prefixes (ng == 0: none)
  const int32_t* slen; // [ng]
  const float* slopes; // [Hq] or nullptr
  float* part_o;       // [T * Hq, nslots, D]; nullptr: one launch writes the results
  float* part_lse;     // [T * Hq, nslots], base 2
  uint32_t* status;
  float scale2;        // no cap: scale * log2(e); cap: 2 * scale / cap * log2(e)
  float cap2;          // cap * log2(e), or 0
  float raw2;          // scale * log2(e)
  float inv_cap2;      // 1 / cap2
  float series_max;    // products below this go by the series of tanh: see cap_series
  int S, T, Hq, Hkv, G, k, ng, max_shared, max_seq_len;
  int chunk, nch_max;  // keys of an item; most items along the keys
  int64_t unit;        // the tensor core kernel's rows: elements between them (divides every stride),
  int page_rows, token_rows, head_rows, map_rows;  // strides in rows, and how many there are
  int box, box_align;  // rows of a box of consecutive ones (0: none), and what its first is a multiple of
  int cl;              // blocks of a cluster that share an item's keys (warp-level kernel)
  int finish;          // this launch joins the shared prefix's chunks, in slots 0 .., and writes the results
  int shared_chunk, shared_nch;
  int blocks, most_steps, most_cuts;  // balanced launch (blocks > 0): see Balance
  int rows;            // rows of an item
  int slot0, nslots;   // this launch's first slot of a row's partial results; slots of a row
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// What is done to a product before the softmax, a kernel each: a cap's dozen
// more operations per element would otherwise be paid by all.
enum Change { kScaled = 0, kBiased = 1, kCapped = 2 /* and a bias, if there are slopes */ };

// Three-way maximum; NaN if any is.
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}
__device__ __forceinline__ float max3_abs(float x, float y, float z) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}
// Pairs of fp32 values in one 64-bit register pair, for the packed instructions.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}

__device__ __forceinline__ float min_nan(float x, float y) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

// Products -> capped exponents of 2: cap tanh(u), u = product scale / cap.
// Below |u| = 1/2, where scores nearly always are, y + y u^2 t(u^2) of the
// uncapped exponent y, no special function: off by a few roundings of y itself,
// whatever the cap.  t is the polynomial of four terms that is nearest to
// (tanh(u) / u - 1) / u^2 there (tanh(u) to 2^-25.9, fitted by least squares with
// weights that grow with the error).  A warp goes by it where all its products of
// 32 keys (on tcgen05; of a block's keys otherwise) are below, else by cap_any: 64
// sequences behind 32768 shared take 244 us, 307 with a score past half the cap in
// every 32; by quotients of four to a reciprocal alone, off by 2^-20 of the cap, 241.
constexpr float kSeries = 0.5f;
__device__ __forceinline__ constexpr float tanh_term(int i) {
  constexpr float c[4] = {-0.333331435918808f, 0.13325878977775574f, -0.05304549261927605f, 0.01724149100482464f};
  return c[i];
}
__device__ __forceinline__ uint64_t cap_near(uint64_t x, const AttendArgs& a) {
  const uint64_t y = mul2(x, pair(a.raw2, a.raw2)), u = mul2(y, pair(a.inv_cap2, a.inv_cap2)), w = mul2(u, u);
  uint64_t t = pair(tanh_term(3), tanh_term(3));
#pragma unroll
  for (int i = 2; i >= 0; --i) t = fma2(w, t, pair(tanh_term(i), tanh_term(i)));
  return fma2(mul2(y, w), t, y);
}
__device__ __forceinline__ void cap_series(float& x0, float& x1, const AttendArgs& a) {
  unpair(cap_near(pair(x0, x1), a), x0, x1);
}
// Any two products of one row: the same, to the bit, below series_max, and
// cap - 2 cap / (e^{2u} + 1) beyond, exact at both ends and off by up to 2^-20 of
// the cap between (near 0 that would be more than the score).  The two quotients
// share a reciprocal (1 / x = y / (x y)), so a NaN of one may reach the other but
// no other row; e^{2u} is held at 2^60, so that the product stays in range.
// Places that a row does not see hold 0 here.
__device__ __forceinline__ void cap_any(float& x0, float& x1, const AttendArgs& a) {
  float n0, n1, y0, y1, e0, e1;
  unpair(cap_near(pair(x0, x1), a), n0, n1);
  unpair(mul2(pair(x0, x1), pair(a.scale2, a.scale2)), y0, y1);
  unpair(add2(pair(ex2(min_nan(y0, 60.f)), ex2(min_nan(y1, 60.f))), pair(1.f, 1.f)), e0, e1);
  const float r = rcp(e0 * e1) * (-2.f * a.cap2);
  x0 = fabsf(x0) < a.series_max ? n0 : fmaf(r, e1, a.cap2);
  x1 = fabsf(x1) < a.series_max ? n1 : fmaf(r, e0, a.cap2);
}

// What a row's exponents are taken from, given its maximum (or, on tcgen05, what
// stands for it).  fp16 holds full precision down to 2^-14 only, so its weights
// are kept up to 2^15 instead of 1: kAbove more than that maximum lets them grow
// to.  A weight of 2^-29 of the largest then still rounds by half a step (2^-21
// on tcgen05, whose rows may outgrow their reference by 2^8), where without it
// 100000 weights of 2^-23.4, 1% of the mass, were off by a third each.  Maxima
// past 2^20 have no bits left for it.  The sum takes the same weights, so the
// results do not depend on it.
template <typename E, int kAbove>
__device__ __forceinline__ float reference(float m) {
  if constexpr (std::is_same<E, __half>::value) return fabsf(m) < 1048576.f ? m - (15 - kAbove) : m;
  return m;
}

// The logarithm of a row's sum l, taken from such a reference.  What fp16's weights
// are raised by is taken out first: lg2's error grows with its result.
template <typename E, int kAbove>
__device__ __forceinline__ float log_sum(float ref, float l) {
  if constexpr (std::is_same<E, __half>::value) return (ref + (15 - kAbove)) + lg2(l * (1.f / (1 << (15 - kAbove))));
  return ref + lg2(l);
}

// Row of the cache seen as [map_rows, D], head 0, or -1: place `off` of page `pg`, or, packed,
// token `pos` of the sequence whose first is `first`.
__device__ __forceinline__ int cache_unit(const AttendArgs& a, int64_t first, int pos, int pg, int off) {
  if (a.c.table) return pg < 0 || pg >= a.c.num_pages ? -1 : pg * a.page_rows + off * a.token_rows;
  const int64_t r = first + pos;
  return r >= 0 && r < a.c.total_keys ? (int)r * a.token_rows : -1;
}

// Tokens of sequence s, at most what the launch was sized for.
__device__ __forceinline__ int seq_len(const AttendArgs& a, int s) {
  const int64_t len = __ldg(a.c.ko + s + 1) - __ldg(a.c.ko + s);
  return len < 0 ? 0 : (int)(len < a.max_seq_len ? len : a.max_seq_len);
}

// Shared tokens of group g, cut to what its first sequence has and to max_shared.
__device__ __forceinline__ int shared_len(const AttendArgs& a, int g) {
  const int s0 = __ldg(a.so + g);
  if (s0 < 0 || s0 >= a.S) return 0;
  return max(0, min(__ldg(a.slen + g), min(a.max_shared, seq_len(a, s0))));
}

// Flags lengths that shared_len cuts; by the threads of one block.  A group
// without sequences has no first one to measure its length by, and nobody reads it.
__device__ __forceinline__ void check_shared(const AttendArgs& a) {
  for (int g = threadIdx.x; g < a.ng; g += blockDim.x)
    if (__ldg(a.so + g) < __ldg(a.so + g + 1) && __ldg(a.slen + g) != shared_len(a, g))
      set_status(a.status, MISA_STATUS_BAD_INPUT);
}

// The group of sequence s, or -1.
__device__ __forceinline__ int group_of(const AttendArgs& a, int s) {
  if (a.ng == 0 || s < __ldg(a.so) || s >= __ldg(a.so + a.ng)) return -1;
  return upper_segment<int32_t>(a.so, a.ng, s);
}

__device__ __forceinline__ int prefix_of(const AttendArgs& a, int s) {
  const int g = group_of(a, s);
  return g < 0 ? 0 : shared_len(a, g);
}

// Items along the keys: own mode at least one (a row that sees nothing is
// written by it), shared mode none for an empty prefix.
__device__ __forceinline__ int own_chunks(const AttendArgs& a, int s, int chunk, int nch_max) {
  if (nch_max == 1) return 1;
  const int own = seq_len(a, s) - prefix_of(a, s);
  return min(nch_max, max(1, (max(own, 0) + chunk - 1) / chunk));
}
__device__ __forceinline__ int shared_chunks(const AttendArgs& a, int g, int chunk, int nch_max) {
  return min(nch_max, (shared_len(a, g) + chunk - 1) / chunk);
}

// Chunks of the shared prefix that sequence s has partial rows of.
__device__ __forceinline__ int shared_slots(const AttendArgs& a, int s) {
  const int g = group_of(a, s);
  return g < 0 ? 0 : shared_chunks(a, g, a.shared_chunk, a.shared_nch);
}

// Query rows of group g (its sequences' queries are consecutive).
__device__ __forceinline__ int2 group_queries(const AttendArgs& a, int g) {
  const int lo = max(0, min(__ldg(a.so + g), a.S)), hi = max(lo, min(__ldg(a.so + g + 1), a.S));
  return make_int2(__ldg(a.qo + lo), __ldg(a.qo + hi));
}

// One work item: rows r0 .. r0+nrows-1 of one key head, row r being query
// qb + r / G, head h * G + r % G; keys [k0, k1) of sequence seq (in selected
// mode: entries [k0, k1) of the query's list).
struct Item {
  int seq, qb, r0, nrows, h, k0, k1, slot;
};

// The items of own and shared mode run over units (sequences or groups), in
// each over row tiles of `rows`, in each over the chunks of its keys, and
// innermost over the key heads.  Their count per unit follows from device
// data, so that every block adds it up for itself: thread i for the i-th
// stretch of units, then a scan.  sums[i] is the count before stretch i,
// sums[n] (returned) all of them.
template <int MODE>
__device__ __forceinline__ int unit_items(const AttendArgs& a, int u, int rows) {
  const int2 q = MODE == kOwn ? make_int2(__ldg(a.qo + u), __ldg(a.qo + u + 1)) : group_queries(a, u);
  const int tiles = (int)(((int64_t)max(0, min(q.y, a.T) - q.x) * a.G + rows - 1) / rows);
  return tiles == 0 ? 0
         : tiles * (MODE == kOwn ? own_chunks(a, u, a.chunk, a.nch_max)
                                 : shared_chunks(a, u, a.chunk, a.nch_max));
}

// sums: kScan + 1 + kScan / 32 ints; every thread of the block (at least
// kScan of them) calls this.
constexpr int kScan = 128;

template <int MODE>
__device__ __forceinline__ int count_items(const AttendArgs& a, int rows, int* sums) {
  const int units = MODE == kOwn ? a.S : a.ng;
  const int per = (units + kScan - 1) / kScan;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int n = 0, x = 0;
  if (threadIdx.x < kScan) {
    for (int u = threadIdx.x * per; u < min(units, ((int)threadIdx.x + 1) * per); ++u)
      n += unit_items<MODE>(a, u, rows);
    x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sums[kScan + 1 + warp] = x;
  }
  __syncthreads();
  if (threadIdx.x < kScan) {
    for (int w = 0; w < warp; ++w) x += sums[kScan + 1 + w];
    sums[threadIdx.x] = x - n;
    if (threadIdx.x == kScan - 1) sums[kScan] = x;
  }
  __syncthreads();
  return sums[kScan];
}

// The unit of item `i` of those that count_items counted, and the items before it.
template <int MODE>
__device__ __forceinline__ int find_unit(const AttendArgs& a, int rows, const int* sums, int i, int& before) {
  const int units = MODE == kOwn ? a.S : a.ng;
  const int per = (units + kScan - 1) / kScan;
  int u = upper_segment<int>(sums, kScan, i) * per;
  before = sums[u / per];
  for (;; ++u) {
    const int n = unit_items<MODE>(a, u, rows);
    if (i - before < n || u + 1 >= units) return u;
    before += n;
  }
}

// Item `i` (without the head) of unit u, the items before whose are counted off.
template <int MODE>
__device__ __forceinline__ void item_of_unit(const AttendArgs& a, int rows, int u, int i, Item& it) {
  const int2 q = MODE == kOwn ? make_int2(__ldg(a.qo + u), __ldg(a.qo + u + 1)) : group_queries(a, u);
  const int nch = MODE == kOwn ? own_chunks(a, u, a.chunk, a.nch_max)
                               : shared_chunks(a, u, a.chunk, a.nch_max);
  const int all = max(0, min(q.y, a.T) - q.x) * a.G;
  const int tiles = (all + rows - 1) / rows;
  // the last row tiles see the most keys: they start first
  const int tile = nch == 1 ? tiles - 1 - i : tiles - 1 - i / nch, c = nch == 1 ? 0 : i % nch;
  it.qb = q.x;
  it.r0 = tile * rows;
  it.nrows = min(rows, all - it.r0);
  it.slot = a.slot0 + c;
  const int lo = MODE == kOwn ? prefix_of(a, u) : 0;
  const int hi = MODE == kOwn ? seq_len(a, u) : shared_len(a, u);
  it.seq = MODE == kOwn ? u : __ldg(a.so + u);
  it.k0 = min(hi, lo + c * a.chunk);
  it.k1 = c == nch - 1 ? hi : min(hi, lo + (c + 1) * a.chunk);
}

// Item `i` (without the head) of those that count_items counted; every thread
// finds the same one.
template <int MODE>
__device__ __forceinline__ void find_item(const AttendArgs& a, int rows, const int* sums, int i, Item& it) {
  int before;
  const int u = find_unit<MODE>(a, rows, sums, i, before);
  item_of_unit<MODE>(a, rows, u, i - before, it);
}

// The same for up to 32 units, by each warp for itself, without count_items:
// a launch of a few microseconds spends less on it than on two barriers.
template <int MODE>
__device__ __forceinline__ int count_few(const AttendArgs& a, int rows) {
  const int lane = threadIdx.x & 31;
  return __reduce_add_sync(0xffffffffu, lane < (MODE == kOwn ? a.S : a.ng) ? unit_items<MODE>(a, lane, rows) : 0);
}
template <int MODE>
__device__ __forceinline__ void find_few(const AttendArgs& a, int rows, int i, Item& it) {
  const int lane = threadIdx.x & 31;
  const int n = lane < (MODE == kOwn ? a.S : a.ng) ? unit_items<MODE>(a, lane, rows) : 0;
  int x = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  const int u = __popc(__ballot_sync(0xffffffffu, x <= i));  // units that end before item i
  item_of_unit<MODE>(a, rows, u, i - __shfl_sync(0xffffffffu, x - n, u & 31), it);
}

// A balanced launch (own mode): the steps of `chunk` keys of all row tiles and
// heads stand in one line, which the blocks cut into equal parts, so that all
// end together whatever the lengths.  A part may begin or end inside a row
// tile's keys, whose partial rows then have a slot for each block that shares
// them: no more than most_cuts + 2, since a part is at least most_steps /
// most_cuts long.
struct Balance {
  int64_t all;  // steps
  int blocks;   // that share them
  __device__ __forceinline__ Balance(const AttendArgs& a, int total) : all((int64_t)total * a.Hkv) {
    const int64_t most = min(all, all * a.most_cuts / a.most_steps);  // no block without a step
    blocks = (int)(most < 1 ? 1 : most < a.blocks ? most : a.blocks);
  }
  __device__ __forceinline__ int64_t begin(int b) const { return b * all / blocks; }
  __device__ __forceinline__ int block_of(int64_t step) const { return (int)(((step + 1) * blocks - 1) / all); }
};

// The item that begins at step `at` and goes to its row tile's end or to step `end`; returns its steps.
__device__ __forceinline__ int find_balanced(const AttendArgs& a, const Balance& bal, int rows, const int* sums,
                                             int64_t at, int64_t end, int block, Item& it) {
  int before;
  const int u = find_unit<kOwn>(a, rows, sums, (int)(at / a.Hkv), before);
  const int first = __ldg(a.qo + u), all = max(0, min(__ldg(a.qo + u + 1), a.T) - first) * a.G;
  const int steps = own_chunks(a, u, a.chunk, a.nch_max);
  const int rem = (int)(at - (int64_t)before * a.Hkv), k = rem % steps, line = rem / steps;
  const int tile = line / a.Hkv;
  it.h = line % a.Hkv;
  it.seq = u;
  it.qb = first;
  it.r0 = tile * rows;
  it.nrows = min(rows, all - it.r0);
  const int n = (int)min((int64_t)(steps - k), end - at);
  const int lo = prefix_of(a, u), hi = seq_len(a, u);
  it.k0 = min(hi, lo + k * a.chunk);
  it.k1 = k + n == steps ? hi : min(hi, lo + (k + n) * a.chunk);
  it.slot = a.slot0 + block - bal.block_of(at - k);
  return n;
}

// Partial rows that a balanced launch left for row (t, head hq) of sequence u.
__device__ __forceinline__ int balanced_slots(const AttendArgs& a, const int* sums, int u, int t, int hq) {
  const Balance bal(a, sums[kScan]);
  const int per = (a.S + kScan - 1) / kScan;
  int before = sums[u / per];
  for (int v = u / per * per; v < u; ++v) before += unit_items<kOwn>(a, v, a.rows);
  const int steps = own_chunks(a, u, a.chunk, a.nch_max);
  const int tile = ((t - __ldg(a.qo + u)) * a.G + hq % a.G) / a.rows;
  const int64_t at = (int64_t)before * a.Hkv + ((int64_t)tile * a.Hkv + hq / a.G) * steps;
  return bal.block_of(at + steps - 1) - bal.block_of(at) + 1;
}

// Selected mode: items run over the queries, their row tiles, the chunks of
// their lists, and innermost over the key heads.  False: a padding row.
__device__ __forceinline__ bool find_selected(const AttendArgs& a, int rows, int i, Item& it) {
  const int tiles = (a.G + rows - 1) / rows;
  const int c = i % a.nch_max;
  i /= a.nch_max;
  const int tile = i % tiles;
  it.qb = i / tiles;
  it.r0 = tile * rows;
  it.nrows = min(rows, a.G - it.r0);
  it.slot = a.slot0 + c;
  it.k0 = c * a.chunk;
  it.k1 = min(a.k, it.k0 + a.chunk);
  const int live = __ldg(a.qo + a.S);
  it.seq = warp_segment(a.qo, a.S, it.qb);
  return it.qb < live;
}

// Position of query t, or -1 (flagged) where it is outside its sequence.
__device__ __forceinline__ int checked_pos(const AttendArgs& a, int t, int seq) {
  const int pos = __ldg(a.q_pos + t);
  if (pos < 0 || pos >= seq_len(a, seq)) {
    set_status(a.status, MISA_STATUS_BAD_INPUT);
    return -1;
  }
  return pos;
}

// Values that no row may take from a masked place.  A weight of 0 times an
// infinity is a NaN, so of keys that only some rows of an item see (those
// behind `near`, its nearest position) what is not finite is cut out of the
// tile, and `poison` gives it back to the rows that do see the key.
// Returns the word without its elements that are not finite.
template <typename E>
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
  constexpr uint32_t M = std::is_same<E, __half>::value ? 0x7c00u : 0x7f80u;
  if ((w & M) == M) w &= 0xffff0000u;
  if ((w & (M << 16)) == (M << 16)) w &= 0x0000ffffu;
  return w;
}
template <typename E>
__device__ __forceinline__ bool cut_infinite(uint4* p) {
  const uint4 x = *p;
  const uint4 y = make_uint4(finite2<E>(x.x), finite2<E>(x.y), finite2<E>(x.z), finite2<E>(x.w));
  if (x.x == y.x && x.y == y.y && x.z == y.z && x.w == y.w) return false;
  *p = y;
  return true;
}
// Adds to o what is not finite of dims [d0, d0 + N) of keys [k0, k1]; N % 8 == 0.
template <typename E, int N>
__device__ __noinline__ void poison(const AttendArgs& a, int seq, int h, int d0, int k0, int k1, float* o) {
  for (int j = k0; j <= k1; ++j) {
    const int64_t r = cache_row(a.c, seq, j);
    if (r < 0) continue;
    const uint16_t* v = a.c.v + r + h * a.c.head_stride + d0;
    for (int d = 0; d < N; ++d) {
      const float x = to_float(__ldg(v + d), E());
      if (!(fabsf(x) < INFINITY)) o[d] += x;
    }
  }
}

// attend_tc.cu: items of 128 rows (split) or 256 (pair) on tcgen05.
int launch_attend_tc(const AttendArgs& a, int mode, int rows, int dtype, int D, int64_t bound, cudaStream_t st);

}  // namespace misa
