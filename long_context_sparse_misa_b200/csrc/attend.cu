// Attention over the key/value cache for few rows per key head (decode), by
// warp-level matrix instructions, and the joining of partial results.
//
//     x = change(q . k) - slope (pos_q - pos_k),  out = sum 2^(x - m) v / sum 2^(x - m)
// in one pass over the keys with the running maximum m and sum of each row.
//
// A block of four warps takes 16 WM rows of one key head against one chunk of
// keys.  WM warps stand side by side over the rows; the 4 / WM groups of them
// take the chunk's key blocks in turn, each with its own shared-memory ring
// filled by cp.async (16-byte chunks, so that any page size, stride or
// selection is read row by row; rows that do not exist are zero-filled, so
// that nothing a masked place holds reaches a product).  The groups' partial
// rows are joined in shared memory.  Up to eight chunks of a row tile are a
// cluster, which joins them over distributed shared memory, with what the
// shared prefix's launch left for the row, and writes the result; more chunks
// leave partial rows in the workspace for combine_kernel.
// Own keys may also be cut into equal parts over all blocks (Balance).
// Bound by HBM where the keys are long (16 sequences of 32768, 8 heads: 231 us,
// 6.4 TB/s), by the chain of dependent loads and joins where they are short
// (one of 1000: 10.1 us).  Two blocks an SM, 16-key blocks for heads of 128: the
// ring's 96 KB keep 64 KB of rows in flight each.
#include "attend.cuh"

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <numeric>

namespace misa {

bool aligned(const void* p, size_t a);                            // abi.cu
int check_ptr(const void* ptr, size_t align, const char* name);  // abi.cu

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;
// Rows of a unit from which the tcgen05 kernel is used, however few the keys (one
// sequence, eight key heads of 128, us of this kernel / of tcgen05):
//   rows    64 keys      128        1024       4096       16384
//    32    9.0 / 16.5  10 / 11   13 / 16    21 / 19    32 / 30
//    48   10.4 / 17.9  13 / 12   16 / 17    30 / 21    43 / 31
//   128   11.5 / 24.1  14 / 17   21 / 24    38 / 28    69 / 37
//   256   11.5 / 32.4  14 / 26   26 / 37    42 / 40   115 / 53
// 300 lists of 256: 32 rows 22 / 24, 48 rows 33 / 26; of 2048: 112 / 90, 171 / 91.
// Below about 1000 keys a rule on the keys too would do better.
constexpr int kTcRows = 48;

template <int D, int WM, int KB>
struct Shape {
  static constexpr int rows = 16 * WM;
  static constexpr int groups = kWarps / WM;
  static constexpr int row_bytes = D * 2;
  static constexpr int half = KB * row_bytes;             // keys or values of a stage
  static constexpr int stage = 2 * half;
  static constexpr int ring = groups * kStages * stage;
  static constexpr int q_bytes = rows * row_bytes;
  static constexpr int merge = groups * rows * (D + 4) * 4;
  static constexpr int big = ring > merge ? ring : merge;
  // q | ring (later the groups' partial rows) | key positions | stage flags | row positions | m, l | scan
  static constexpr int bytes = q_bytes + big + groups * kStages * KB * 4 + groups * kStages * 4 * WM + rows * 4 +
                               groups * rows * 8 + rows * 4 + (kScan + 1 + kScan / 32) * 4 + 16 + 64;
};

constexpr int resident_blocks(int bytes) {
  return bytes <= 0 ? 1 : std::max(1, std::min(8, 227 * 1024 / (bytes + 1024)));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                         __nv_bfloat16) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __half) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The warps of one key group (WM of them) wait for one another.
template <int WM>
__device__ __forceinline__ void group_sync(int group) {
  if constexpr (WM == 1) {
    __syncwarp();
  } else {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(WM * 32) : "memory");
  }
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// Reads of block `rank`'s shared memory; without a cluster the block's own.
__device__ __forceinline__ uint32_t cluster_at(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr, int rank) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(cluster_at(addr, rank)));
  return x;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr, int rank) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(cluster_at(addr, rank)));
  return x;
}

// Keys [k0, k1) of an item, or the part of them that block `rank` of its cluster takes.
__device__ __forceinline__ int2 part_of(const AttendArgs& a, int k0, int k1, int rank, int block) {
  if (a.cl == 1) return make_int2(k0, k1);
  const int shift = a.cl == 2 ? 1 : a.cl == 4 ? 2 : 3;
  const int per = (((max(k1 - k0, 0) + a.cl - 1) >> shift) + block - 1) / block * block;
  return make_int2(k0 + rank * per, min(k1, k0 + (rank + 1) * per));
}

// Row r of an item among all [T, Hq].
__device__ __forceinline__ int64_t row_of_item(const AttendArgs& a, const Item& it, int r) {
  const int g = it.r0 + r;
  return (int64_t)(it.qb + g / a.G) * a.Hq + it.h * a.G + g % a.G;
}

template <typename E>
__device__ __forceinline__ uint4 pack8(const float (&x)[8], E tag) {
  return make_uint4(pack2(x[0], x[1], tag), pack2(x[2], x[3], tag), pack2(x[4], x[5], tag), pack2(x[6], x[7], tag));
}

// MODE: which keys; KIND: what is done to the products (Change).
template <typename E, int D, int WM, int KB, int MODE, int KIND>
__global__ void __launch_bounds__(kThreads) attend_kernel(const __grid_constant__ AttendArgs a) {
  pdl_wait_then_release();
  using Sh = Shape<D, WM, KB>;
  constexpr int kChunks = D / 8;         // 16-byte chunks of a row
  constexpr int kNT = KB / 8, kDT = D / 8;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* s_q = smem;
  uint8_t* s_ring = s_q + Sh::q_bytes;
  int* s_key = reinterpret_cast<int*>(s_ring + Sh::big);
  int* s_mask = s_key + Sh::groups * kStages * KB;
  int* s_pos = s_mask + Sh::groups * kStages * WM;
  float* s_ml = reinterpret_cast<float*>(s_pos + Sh::rows);
  float* s_lse = s_ml + Sh::groups * Sh::rows * 2;
  int* s_sum = reinterpret_cast<int*>(s_lse + Sh::rows);

  volatile int* s_cut = s_sum + kScan + 1 + kScan / 32;  // something was cut out of a value block

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wm = warp % WM, grp = warp / WM;
  const E tag = E();

  if (MODE == kShared && blockIdx.x == 0) check_shared(a);
  const bool few = (MODE == kOwn ? a.S : a.ng) <= 32 && a.blocks == 0;
  int total = 0;
  if constexpr (MODE == kSelected) {
    total = a.T * ((a.G + Sh::rows - 1) / Sh::rows) * a.nch_max;
  } else if (few) {
    total = count_few<MODE>(a, Sh::rows);
  } else {
    total = count_items<MODE>(a, Sh::rows, s_sum);
  }
  const int rank = a.cl > 1 ? (int)cluster_rank() : 0;
  int64_t w = blockIdx.x / a.cl, end = (int64_t)total * a.Hkv;
  Balance bal(a, total);
  const bool balanced = MODE == kOwn && a.blocks > 0;
  if (balanced) {
    w = (int)blockIdx.x < bal.blocks ? bal.begin(blockIdx.x) : 0;
    end = (int)blockIdx.x < bal.blocks ? bal.begin(blockIdx.x + 1) : 0;
  }
  while (w < end) {
    Item it;
    if constexpr (MODE == kSelected) {
      it.h = (int)(w % a.Hkv);
      const bool live = find_selected(a, Sh::rows, (int)(w / a.Hkv), it);
      w += gridDim.x / a.cl;
      if (!live) continue;
    } else if (balanced) {
      w += find_balanced(a, bal, Sh::rows, s_sum, w, end, blockIdx.x, it);
    } else {
      it.h = (int)(w % a.Hkv);
      if (few) find_few<MODE>(a, Sh::rows, (int)(w / a.Hkv), it);
      else find_item<MODE>(a, Sh::rows, s_sum, (int)(w / a.Hkv), it);
      w += gridDim.x / a.cl;
    }
    __syncthreads();  // the previous item is done with shared memory

    // A list's first entries are read ahead of everything else: they lead to the pages, those to the rows.
    int ahead[2] = {-1, -1};
    if constexpr (MODE == kSelected) {
      const int2 part = part_of(a, it.k0, it.k1, rank, KB);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int j = part.x + (grp + i * Sh::groups) * KB + lane;
        if (lane < KB && j < part.y) ahead[i] = __ldg(a.idx + (int64_t)it.qb * a.k + j);
      }
    }
    if (threadIdx.x == 0) *s_cut = 0;
    // Rows: their q, swizzled, and their queries' positions (-1 sees nothing).
    constexpr int kQ = Sh::rows * kChunks / kThreads;
    uint4 qv[kQ];
#pragma unroll
    for (int u = 0; u < kQ; ++u) {
      const int i = threadIdx.x + u * kThreads, r = i / kChunks;
      qv[u] = make_uint4(0, 0, 0, 0);
      if (r < it.nrows) qv[u] = __ldg(reinterpret_cast<const uint4*>(a.q + row_of_item(a, it, r) * D) + i % kChunks);
    }
    for (int r = threadIdx.x; r < Sh::rows; r += kThreads) {
      int pos = -1;
      if (r < it.nrows) {
        const int t = it.qb + (it.r0 + r) / a.G;
        int sq = it.seq;
        if (MODE == kShared) sq = upper_segment<int32_t>(a.qo, a.S, t);
        pos = checked_pos(a, t, sq);
      }
      s_pos[r] = pos;
    }
#pragma unroll
    for (int u = 0; u < kQ; ++u) {
      const int i = threadIdx.x + u * kThreads, r = i / kChunks, c = i % kChunks;
      *reinterpret_cast<uint4*>(s_q + r * Sh::row_bytes + ((c ^ (r & 7)) << 4)) = qv[u];
    }
    __syncthreads();
    // Furthest and nearest position of the real rows; least: of those that see anything.
    int far = -1, near = 0x7fffffff, least = 0x7fffffff;
    for (int r = lane; r < it.nrows; r += 32) {
      const int pos = s_pos[r];
      far = max(far, pos);
      near = min(near, pos);
      if (pos >= 0) least = min(least, pos);
    }
    far = __reduce_max_sync(0xffffffffu, far);
    near = __reduce_min_sync(0xffffffffu, near);
    least = __reduce_min_sync(0xffffffffu, least);
    // this block's keys: the item's, or its part of the cluster's
    const int2 part = part_of(a, it.k0, MODE == kSelected ? it.k1 : min(it.k1, far + 1), rank, KB);
    const int k0 = part.x, k1 = part.y;
    const int nblk = k1 > k0 ? (k1 - k0 + KB - 1) / KB : 0;
    const int mine = nblk > grp ? (nblk - grp + Sh::groups - 1) / Sh::groups : 0;  // blocks of this group

    uint32_t fq[D / 16][4];
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      const int r = wm * 16 + (lane & 15), c = ks * 2 + (lane >> 4);
      ldsm4(fq[ks], smem_u32(s_q + r * Sh::row_bytes + ((c ^ (r & 7)) << 4)));
    }
    const int row0 = wm * 16 + (lane >> 2), row1 = row0 + 8;
    const int pos0 = s_pos[row0], pos1 = s_pos[row1];
    float sl0 = 0.f, sl1 = 0.f;
    const bool bias = KIND == kBiased || (KIND == kCapped && a.slopes);
    if (bias) {
      sl0 = row0 < it.nrows ? __ldg(a.slopes + it.h * a.G + (it.r0 + row0) % a.G) * kLog2e : 0.f;
      sl1 = row1 < it.nrows ? __ldg(a.slopes + it.h * a.G + (it.r0 + row1) % a.G) * kLog2e : 0.f;
    }

    // Lane l knows key l of a block: its position and where its row is.
    const int64_t head = it.h * a.c.head_stride;
    auto key_of = [&](int i) -> int {  // position of this lane's key in the group's i-th block, -1: none
      const int j = k0 + (grp + i * Sh::groups) * KB + lane;
      if (i >= mine || lane >= KB || j >= k1) return -1;
      if constexpr (MODE == kSelected) return __ldg(a.idx + (int64_t)it.qb * a.k + j);
      return j;
    };
    auto row_of = [&](int key) -> int64_t {
      if (MODE == kSelected && key > far) {
        // beyond the query's position, or a query that sees nothing
        if (far >= 0) set_status(a.status, MISA_STATUS_BAD_INPUT);
        return -1;
      }
      if (key < 0) return -1;
      const int64_t r = cache_row(a.c, it.seq, key);
      if (r < 0) set_status(a.status, MISA_STATUS_BOUNDS);
      return r;
    };
    uint8_t* ring = s_ring + grp * kStages * Sh::stage;
    int* keys = s_key + grp * kStages * KB;
    int* masks = s_mask + (grp * kStages) * WM;
    auto load = [&](int i, int key, int64_t row) {
      const int st = i % kStages;
      uint8_t* dst = ring + st * Sh::stage;
      constexpr int per = 32 / kChunks;  // rows of one copy instruction
      constexpr int share = KB / WM;     // rows that this warp copies
      const int c = lane % kChunks;
      if (i < mine) {
#pragma unroll
        for (int u = 0; u < share / per; ++u) {
          const int r = wm * share + u * per + lane / kChunks;
          const int64_t off = __shfl_sync(0xffffffffu, row, r);
          const int64_t e = (off < 0 ? 0 : off) + head + c * 8;
          uint8_t* d = dst + r * Sh::row_bytes + ((c ^ (r & 7)) << 4);
          cp_async_16(d, a.c.k + e, off >= 0);
          cp_async_16(d + Sh::half, a.c.v + e, off >= 0);
        }
        if (wm == 0 && lane < KB) keys[st * KB + lane] = row < 0 ? -1 : key;
        // 1: a key of the block needs a mask; 2: some rows see it, others not
        const bool mask = !__all_sync(0xffffffffu, lane >= KB || (row >= 0 && key <= near));
        const bool part = MODE != kSelected && __any_sync(0xffffffffu, lane < KB && row >= 0 && key > least);
        if (lane == 0) masks[st * WM + wm] = part ? 2 : mask;
      }
      cp_async_commit();
    };

    float o[kDT][4];
#pragma unroll
    for (int n = 0; n < kDT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[n][j] = 0.f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

    // kStages - 1 blocks in flight; positions two blocks ahead of the copies, rows one.
    int key_a = MODE == kSelected ? ahead[0] : key_of(0);
    int64_t row_a = row_of(key_a);
    int key_b = MODE == kSelected ? ahead[1] : key_of(1);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      const int64_t row_b = row_of(key_b);
      const int key_c = key_of(i + 2);
      load(i, key_a, row_a);
      key_a = key_b;
      row_a = row_b;
      key_b = key_c;
    }
    for (int i = 0; i < mine; ++i) {
      cp_async_wait_group<kStages - 2>();
      group_sync<WM>(grp);
      {
        const int64_t row_b = row_of(key_b);
        const int key_c = key_of(i + kStages + 1);
        load(i + kStages - 1, key_a, row_a);
        key_a = key_b;
        row_a = row_b;
        key_b = key_c;
      }
      const int st = i % kStages;
      const uint32_t kb = smem_u32(ring + st * Sh::stage), vb = kb + Sh::half;
      float s[kNT][4];
#pragma unroll
      for (int n = 0; n < kNT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[n][j] = 0.f;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
#pragma unroll
        for (int n = 0; n < kNT; n += 2) {
          uint32_t b[4];
          const int r = n * 8 + ((lane >> 4) << 3) + (lane & 7), c = ks * 2 + ((lane >> 3) & 1);
          ldsm4(b, kb + r * Sh::row_bytes + ((c ^ (r & 7)) << 4));
          mma16816(s[n], fq[ks], b[0], b[1], tag);
          mma16816(s[n + 1], fq[ks], b[2], b[3], tag);
        }
      }
      const int mask = masks[st * WM + wm];
      if (MODE != kSelected && mask == 2) {
        bool cut = false;
        for (int i = wm * 32 + lane; i < KB * kChunks; i += WM * 32) {
          const int r = i / kChunks, c = i % kChunks;
          if (keys[st * KB + r] > least)
            cut |= cut_infinite<E>(reinterpret_cast<uint4*>(ring + st * Sh::stage + Sh::half + r * Sh::row_bytes +
                                                           ((c ^ (r & 7)) << 4)));
        }
        if (cut) *s_cut = 1;
        group_sync<WM>(grp);
      }
      if constexpr (KIND == kCapped) {
        float most = 0.f;
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          if (mask) {
            const int2 kp = *reinterpret_cast<const int2*>(keys + st * KB + n * 8 + (lane & 3) * 2);
            if (kp.x < 0 || kp.x > pos0) s[n][0] = 0.f;
            if (kp.y < 0 || kp.y > pos0) s[n][1] = 0.f;
            if (kp.x < 0 || kp.x > pos1) s[n][2] = 0.f;
            if (kp.y < 0 || kp.y > pos1) s[n][3] = 0.f;
          }
          most = max3_abs(max3_abs(most, s[n][0], s[n][1]), s[n][2], s[n][3]);
        }
        if (__all_sync(0xffffffffu, most < a.series_max)) {
#pragma unroll
          for (int j = 0; j < 2 * kNT; ++j) cap_series(s[j >> 1][(j & 1) * 2], s[j >> 1][(j & 1) * 2 + 1], a);
        } else {
#pragma unroll
          for (int j = 0; j < 2 * kNT; ++j) cap_any(s[j >> 1][(j & 1) * 2], s[j >> 1][(j & 1) * 2 + 1], a);
        }
      }
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        if constexpr (KIND != kCapped) {
#pragma unroll
          for (int j = 0; j < 4; ++j) s[n][j] *= a.scale2;
        }
        if (bias || mask) {
          const int2 kp = *reinterpret_cast<const int2*>(keys + st * KB + n * 8 + (lane & 3) * 2);
          if (bias) {
            s[n][0] = fmaf(-sl0, (float)(pos0 - kp.x), s[n][0]);
            s[n][1] = fmaf(-sl0, (float)(pos0 - kp.y), s[n][1]);
            s[n][2] = fmaf(-sl1, (float)(pos1 - kp.x), s[n][2]);
            s[n][3] = fmaf(-sl1, (float)(pos1 - kp.y), s[n][3]);
          }
          if (mask) {
            if (kp.x < 0 || kp.x > pos0) s[n][0] = -INFINITY;
            if (kp.y < 0 || kp.y > pos0) s[n][1] = -INFINITY;
            if (kp.x < 0 || kp.x > pos1) s[n][2] = -INFINITY;
            if (kp.y < 0 || kp.y > pos1) s[n][3] = -INFINITY;
          }
        }
      }
      float t0 = m0, t1 = m1;
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        t0 = fmaxf(t0, fmaxf(s[n][0], s[n][1]));
        t1 = fmaxf(t1, fmaxf(s[n][2], s[n][3]));
      }
      t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 1));
      t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 1));
      t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, 2));
      t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, 2));
      // a row that has seen nothing yet keeps 0 as its reference: 2^(-inf - 0) = 0
      const float r0 = t0 == -INFINITY ? 0.f : reference<E, 0>(t0), r1 = t1 == -INFINITY ? 0.f : reference<E, 0>(t1);
      if (__any_sync(0xffffffffu, t0 != m0 || t1 != m1)) {
        const float c0 = ex2(reference<E, 0>(m0) - r0), c1 = ex2(reference<E, 0>(m1) - r1);
        l0 *= c0;
        l1 *= c1;
#pragma unroll
        for (int n = 0; n < kDT; ++n) {
          o[n][0] *= c0;
          o[n][1] *= c0;
          o[n][2] *= c1;
          o[n][3] *= c1;
        }
        m0 = t0;
        m1 = t1;
      }
      uint32_t p[kNT / 2][4];
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        s[n][0] = ex2(s[n][0] - r0);
        s[n][1] = ex2(s[n][1] - r0);
        s[n][2] = ex2(s[n][2] - r1);
        s[n][3] = ex2(s[n][3] - r1);
        l0 += s[n][0] + s[n][1];
        l1 += s[n][2] + s[n][3];
        // weights round to the cache's type for the matrix instruction: half a
        // step each, independent, against the output's own single rounding
        p[n / 2][(n & 1) * 2] = pack2(s[n][0], s[n][1], tag);
        p[n / 2][(n & 1) * 2 + 1] = pack2(s[n][2], s[n][3], tag);
      }
#pragma unroll
      for (int kk = 0; kk < KB / 16; ++kk) {
#pragma unroll
        for (int n = 0; n < kDT; n += 2) {
          uint32_t b[4];
          const int r = kk * 16 + (lane & 15), c = n + (lane >> 4);
          ldsm4t(b, vb + r * Sh::row_bytes + ((c ^ (r & 7)) << 4));
          mma16816(o[n], p[kk], b[0], b[1], tag);
          mma16816(o[n + 1], p[kk], b[2], b[3], tag);
        }
      }
    }
    cp_async_wait_group<0>();
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
    __syncthreads();  // every group is done with its ring

    // Join the groups: O in the ring's place, [group][row][D + 4].
    float* s_o = reinterpret_cast<float*>(s_ring);
    {
      float* d0 = s_o + (grp * Sh::rows + row0) * (D + 4) + (lane & 3) * 2;
      float* d1 = d0 + 8 * (D + 4);
#pragma unroll
      for (int n = 0; n < kDT; ++n) {
        *reinterpret_cast<float2*>(d0 + n * 8) = make_float2(o[n][0], o[n][1]);
        *reinterpret_cast<float2*>(d1 + n * 8) = make_float2(o[n][2], o[n][3]);
      }
      if ((lane & 3) == 0) {
        float* ml = s_ml + (grp * Sh::rows) * 2;
        ml[row0 * 2] = reference<E, 0>(m0);
        ml[row0 * 2 + 1] = l0;
        ml[row1 * 2] = reference<E, 0>(m1);
        ml[row1 * 2 + 1] = l1;
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < it.nrows * kChunks; i += kThreads) {
      const int r = i / kChunks, c = i % kChunks;
      float m = -INFINITY;
#pragma unroll
      for (int g = 0; g < Sh::groups; ++g) m = fmaxf(m, s_ml[(g * Sh::rows + r) * 2]);
      const float ref = m == -INFINITY ? 0.f : m;
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, l = 0.f;
#pragma unroll
      for (int g = 0; g < Sh::groups; ++g) {
        const float f = ex2(s_ml[(g * Sh::rows + r) * 2] - ref);
        l = fmaf(f, s_ml[(g * Sh::rows + r) * 2 + 1], l);
        const float4* src = reinterpret_cast<const float4*>(s_o + (g * Sh::rows + r) * (D + 4) + c * 8);
        const float4 x = src[0], y = src[1];
        acc[0] = fmaf(f, x.x, acc[0]);
        acc[1] = fmaf(f, x.y, acc[1]);
        acc[2] = fmaf(f, x.z, acc[2]);
        acc[3] = fmaf(f, x.w, acc[3]);
        acc[4] = fmaf(f, y.x, acc[4]);
        acc[5] = fmaf(f, y.y, acc[5]);
        acc[6] = fmaf(f, y.z, acc[6]);
        acc[7] = fmaf(f, y.w, acc[7]);
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that saw nothing: zeros
      const float lse2 = l == 0.f ? -INFINITY : log_sum<E, 0>(ref, l);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = l == 0.f ? 0.f : acc[j] * inv;
      if (MODE != kSelected && *s_cut && least < s_pos[r])
        poison<E, 8>(a, it.seq, it.h, c * 8, max(k0, least + 1), min(k1 - 1, s_pos[r]), acc);
      if (a.cl > 1 || a.finish) {
        // this block's row, in the place of its first group's
        float4* d = reinterpret_cast<float4*>(s_o + r * (D + 4) + c * 8);
        d[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        d[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if (c == 0) s_lse[r] = lse2;
        continue;
      }
      const int64_t row = row_of_item(a, it, r);
      if (a.part_o) {
        float4* d = reinterpret_cast<float4*>(a.part_o + (row * a.nslots + it.slot) * D + c * 8);
        d[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        d[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if (c == 0) a.part_lse[row * a.nslots + it.slot] = lse2;
      } else {
        *reinterpret_cast<uint4*>(a.out + row * D + c * 8) = pack8(acc, tag);
        if (c == 0 && a.lse) a.lse[row] = lse2 * kLn2;
      }
    }
    if (a.cl > 1 || a.finish) {
      // Join the blocks, and the shared prefix's chunks; the rows are spread over the cluster.
      if (a.cl > 1) cluster_sync();
      else __syncthreads();
      const int n_shared = MODE == kOwn && a.finish ? shared_slots(a, it.seq) : 0;
      for (int i = rank * kThreads + threadIdx.x; i < it.nrows * kChunks; i += a.cl * kThreads) {
        const int r = i / kChunks, c = i % kChunks;
        const int64_t row = row_of_item(a, it, r);
        // The chunk's lanes share the row: lane b reads block b's weight, and all the chunks at once.
        const uint32_t lse_at = smem_u32(s_lse + r), o_at = smem_u32(s_o + r * (D + 4) + c * 8);
        const uint32_t team = (kChunks == 16 ? 0xffffu : 0xffu) << (lane & ~(kChunks - 1));
        float4 ox[8], oy[8];
#pragma unroll
        for (int b = 0; b < 8; ++b)
          if (b < a.cl) {
            ox[b] = ld_cluster4(o_at, b);
            oy[b] = ld_cluster4(o_at + 16, b);
          }
        const float mine_lse = c < a.cl ? ld_cluster(lse_at, c) : -INFINITY;
        const float* pl = a.part_lse + row * a.nslots;
        float m = mine_lse;
        for (int b = c; b < n_shared; b += kChunks) m = fmaxf(m, pl[b]);
#pragma unroll
        for (int o = kChunks / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(team, m, o));
        const float ref = m == -INFINITY ? 0.f : m;
        const float mine_f = ex2(mine_lse - ref);
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, l = 0.f;
        auto take = [&](float f, const float4& x, const float4& y) {
          l += f;
          acc[0] = fmaf(f, x.x, acc[0]);
          acc[1] = fmaf(f, x.y, acc[1]);
          acc[2] = fmaf(f, x.z, acc[2]);
          acc[3] = fmaf(f, x.w, acc[3]);
          acc[4] = fmaf(f, y.x, acc[4]);
          acc[5] = fmaf(f, y.y, acc[5]);
          acc[6] = fmaf(f, y.z, acc[6]);
          acc[7] = fmaf(f, y.w, acc[7]);
        };
#pragma unroll
        for (int b = 0; b < 8; ++b)
          if (b < a.cl) take(__shfl_sync(team, mine_f, b, kChunks), ox[b], oy[b]);
#pragma unroll 4
        for (int b = 0; b < n_shared; ++b) {
          const float4* src = reinterpret_cast<const float4*>(a.part_o + (row * a.nslots + b) * D + c * 8);
          take(ex2(pl[b] - ref), src[0], src[1]);
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] *= inv;
        *reinterpret_cast<uint4*>(a.out + row * D + c * 8) = pack8(acc, tag);
        if (c == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : (ref + lg2(l)) * kLn2;
      }
      if (a.cl > 1) cluster_sync();  // nobody reads this block's rows any more
    }
  }
}

// Joins a row's partial results: the shared prefix's chunks in slots 0 ..,
// the own (or selected) ones from own0 on.  One block of four warps a row;
// warp w takes slots w, w + 4, ..; a fixed order, so the same bits every time.
struct CombineArgs {
  AttendArgs a;
  int own_chunk, own_max, shared_chunk, shared_max, own0;
  bool selected;
};

template <typename E, int D>
__global__ void __launch_bounds__(kThreads) combine_kernel(const __grid_constant__ CombineArgs p) {
  pdl_wait_then_release();
  const AttendArgs& a = p.a;
  __shared__ float s_o[kWarps][D];
  __shared__ float s_l[kWarps];
  __shared__ int s_sum[kScan + 1 + kScan / 32];
  if (a.blocks > 0) count_items<kOwn>(a, a.rows, s_sum);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;
  const int t = (int)(row / a.Hq);
  if (t >= __ldg(a.qo + a.S)) return;
  int n_own = p.own_max, n_shared = 0;
  if (!p.selected) {
    const int seq = warp_segment(a.qo, a.S, t);
    n_own = a.blocks > 0 ? balanced_slots(a, s_sum, seq, t, (int)(row % a.Hq)) : own_chunks(a, seq, p.own_chunk, p.own_max);
    const int g = group_of(a, seq);
    if (g >= 0) n_shared = shared_chunks(a, g, p.shared_chunk, p.shared_max);
  }
  const int n = n_shared + n_own;
  const float* lse = a.part_lse + row * a.nslots;
  auto slot = [&](int i) { return i < n_shared ? i : p.own0 + i - n_shared; };
  float m = -INFINITY;
  bool nan = false;
  for (int i = lane; i < n; i += 32) {
    const float x = lse[slot(i)];
    nan |= x != x;
    m = fmaxf(m, x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (__any_sync(0xffffffffu, nan)) m = __int_as_float(0x7fffffff);
  const float ref = m == -INFINITY ? 0.f : m;
  constexpr int kV = D / 32;  // floats of a lane
  float acc[kV], l = 0.f;
#pragma unroll
  for (int j = 0; j < kV; ++j) acc[j] = 0.f;
  const float* po = a.part_o + row * a.nslots * D + lane * kV;
#pragma unroll 4
  for (int i = warp; i < n; i += kWarps) {
    const int s = slot(i);
    const float f = ex2(lse[s] - ref);
    l += f;
    if constexpr (kV == 4) {
      const float4 x = *reinterpret_cast<const float4*>(po + (int64_t)s * D);
      acc[0] = fmaf(f, x.x, acc[0]);
      acc[1] = fmaf(f, x.y, acc[1]);
      acc[2] = fmaf(f, x.z, acc[2]);
      acc[3] = fmaf(f, x.w, acc[3]);
    } else {
      const float2 x = *reinterpret_cast<const float2*>(po + (int64_t)s * D);
      acc[0] = fmaf(f, x.x, acc[0]);
      acc[1] = fmaf(f, x.y, acc[1]);
    }
  }
#pragma unroll
  for (int j = 0; j < kV; ++j) s_o[warp][lane * kV + j] = acc[j];
  if (lane == 0) s_l[warp] = l;
  __syncthreads();
  l = s_l[0] + s_l[1] + s_l[2] + s_l[3];
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (threadIdx.x < D / 2) {
    const int d = threadIdx.x * 2;
    const float x = (s_o[0][d] + s_o[1][d]) + (s_o[2][d] + s_o[3][d]);
    const float y = (s_o[0][d + 1] + s_o[1][d + 1]) + (s_o[2][d + 1] + s_o[3][d + 1]);
    *reinterpret_cast<uint32_t*>(a.out + row * D + d) = pack2(x * inv, y * inv, E());
  }
  if (threadIdx.x == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : (ref + lg2(l)) * kLn2;
}

template <typename E, int D, int WM, int KB, int MODE, int KIND>
int launch_rows(const AttendArgs& a, int64_t bound, cudaStream_t st) {
  using Sh = Shape<D, WM, KB>;
  auto kern = attend_kernel<E, D, WM, KB, MODE, KIND>;
  int rc = set_smem_limit((const void*)kern, Sh::bytes);
  if (rc) return rc;
  // one wave of resident blocks walks the items; clusters, whose lengths
  // differ, come in several, so that the hardware evens them out
  const int resident = resident_blocks(Sh::bytes);
  const int64_t wave = std::max<int64_t>(1, (int64_t)num_sms() * resident / a.cl * (a.cl > 1 ? 8 : 1));
  const unsigned grid = a.blocks > 0 ? (unsigned)a.blocks : (unsigned)(std::max<int64_t>(1, std::min(bound, wave)) * a.cl);
  static const char* const names[] = {"attend", "attend_shared", "attend_selected"};
  ProfScope ps(names[MODE], st);
  return cuda_fail(a.cl > 1 ? launch_pdl_cluster(kern, dim3(grid), dim3(kThreads), a.cl, Sh::bytes, st, a)
                            : launch_pdl(kern, dim3(grid), dim3(kThreads), Sh::bytes, st, a),
                   "attend_kernel");
}

template <typename E, int D, int WM, int KB, int MODE>
int launch_kind(const AttendArgs& a, int64_t bound, cudaStream_t st) {
  return a.cap2 > 0.f ? launch_rows<E, D, WM, KB, MODE, kCapped>(a, bound, st)
         : a.slopes   ? launch_rows<E, D, WM, KB, MODE, kBiased>(a, bound, st)
                      : launch_rows<E, D, WM, KB, MODE, kScaled>(a, bound, st);
}

template <typename E, int D, int MODE>
int launch_width(const AttendArgs& a, int rows, int64_t bound, cudaStream_t st) {
  // two blocks an SM: one's start and end behind the other's copies
  if (rows == 16) return launch_kind<E, D, 1, D == 128 ? 16 : 32, MODE>(a, bound, st);
  if (rows == 32) return launch_kind<E, D, 2, 32, MODE>(a, bound, st);
  return launch_kind<E, D, 4, 32, MODE>(a, bound, st);
}

template <int MODE>
int launch_attend(const AttendArgs& a, int dtype, int D, bool tc, int rows, int64_t bound, cudaStream_t st) {
  if (tc) return launch_attend_tc(a, MODE, rows, dtype, D, bound, st);
  if (dtype == MISA_BF16)
    return D == 128 ? launch_width<__nv_bfloat16, 128, MODE>(a, rows, bound, st)
                    : launch_width<__nv_bfloat16, 64, MODE>(a, rows, bound, st);
  return D == 128 ? launch_width<__half, 128, MODE>(a, rows, bound, st)
                  : launch_width<__half, 64, MODE>(a, rows, bound, st);
}

int launch_combine(const CombineArgs& c, int dtype, int D, cudaStream_t st) {
  const dim3 grid((unsigned)((int64_t)c.a.T * c.a.Hq));
  ProfScope ps("attend_combine", st);
  cudaError_t e;
  if (dtype == MISA_BF16)
    e = D == 128 ? launch_pdl(combine_kernel<__nv_bfloat16, 128>, grid, dim3(kThreads), 0, st, c)
                 : launch_pdl(combine_kernel<__nv_bfloat16, 64>, grid, dim3(kThreads), 0, st, c);
  else
    e = D == 128 ? launch_pdl(combine_kernel<__half, 128>, grid, dim3(kThreads), 0, st, c)
                 : launch_pdl(combine_kernel<__half, 64>, grid, dim3(kThreads), 0, st, c);
  return cuda_fail(e, "combine_kernel");
}

// How a call is divided: from host-side bounds alone, so that a captured call
// stays right when the device's lengths change within them.
struct Part {
  bool tc = false;     // tcgen05 (attend_tc.cu)
  int rows = 16;       // rows of an item
  int chunk = 1;       // keys of an item
  int nch = 0;         // most items along the keys (0: no launch)
  int cl = 1;          // blocks of a cluster that share an item's keys
  int cuts = 0;        // balanced launch: most_cuts of its blocks (0: not one)
  int64_t bound = 0;   // most items, heads included
};
struct Plan {
  Part own, shared;    // own: the selected launch too
  int nslots = 1;
  bool finish = false;  // the own launch writes the results, with what the shared one left
  bool partial = false;
  size_t o_bytes = 0, lse_bytes = 0;
  size_t bytes() const { return partial ? o_bytes + lse_bytes + 256 : 256; }
};

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// The cache as rows of D elements a fixed step apart, which every stride is a
// multiple of, so that a row has one index in a tensor map.  rows == 0: the
// steps overlap, or there are more rows than an index holds.
struct RowGrid {
  int64_t unit = 0, rows = 0;
};
RowGrid row_grid(const misa_problem_t* p, const misa_kv_cache_t* c) {
  const int64_t n[3] = {c->page_table ? c->num_pages : 1, c->page_table ? c->page_size : p->total_keys,
                        c->num_kv_heads};
  const int64_t step[3] = {c->page_stride, c->token_stride, c->head_stride};
  RowGrid g;
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1) g.unit = std::gcd(g.unit, step[i]);
  if (g.unit == 0) g.unit = c->head_dim;
  int64_t last = 0;
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1) {
      const int64_t s = step[i] / g.unit;
      if (s && n[i] - 1 > (int64_t(1) << 31) / s) return RowGrid();
      last += (n[i] - 1) * s;
    }
  if (g.unit >= c->head_dim && last < (int64_t(1) << 31) - 2 && g.unit < (int64_t(1) << 38)) g.rows = last + 1;
  return g;
}

// Rows of an item for units (sequences, groups, queries) of about `rows` rows.
void pick_rows(Part& p, int64_t rows, bool grid) {
  p.tc = grid && rows >= kTcRows;
  if (p.tc) p.rows = rows > 128 ? 256 : 128;
  else p.rows = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

// Cuts the keys of `units` row tiles (heads included), about `keys` each and
// at most max_keys, so that the launch ends soonest.  Costs are in keys of a
// block (512 bytes at 23 GB/s, 22 ns, in the warp-level kernel): the items fill
// the GPU's places in whole waves, and an item costs its keys and a fixed part;
// a cluster's join little, partial rows through the workspace a second launch
// (9 us).  Own keys may instead be balanced over all blocks: no waves.  The costs
// were measured with heads of 128 and serve heads of 64 unchanged, whose keys are
// half as long: their fixed parts then count for half of what they are.
constexpr int kStep = 128;  // keys of a balanced launch's step
void split_keys(Part& p, int64_t units, int64_t keys, int64_t max_keys, bool clusters, bool balance) {
  const int64_t places = num_sms() * (p.tc ? 1 : 2);
  const int64_t fixed = p.tc ? 512 : 96, least = p.tc ? 256 : 64, join = p.tc ? 512 : 420;
  units = std::max<int64_t>(1, units);
  keys = std::max<int64_t>(1, std::min(keys, max_keys));
  const int64_t most = (keys + least - 1) / least;
  int64_t best = 1, best_cost = INT64_MAX;
  auto consider = [&](int64_t c, bool in_cluster) {
    if (c < 1 || c > most) return;
    const int64_t waves = (units * c + places - 1) / places;
    const int64_t cost = waves * ((keys + c - 1) / c + fixed) + (c == 1 ? 0 : in_cluster ? 64 : join + 8 * c);
    if (cost >= best_cost) return;
    best = c;
    best_cost = cost;
    p.cl = in_cluster ? (int)c : 1;
  };
  consider(1, false);
  for (int c = 2; clusters && c <= 8; c *= 2) consider(c, true);
  if (balance) {
    if ((units * keys + places - 1) / places + (units / places + 2) * fixed + join < best_cost) {
      p.cl = 1;
      p.cuts = (int)std::max<int64_t>(8, (2 * places + units - 1) / units);
      p.chunk = kStep;
      p.nch = p.cuts + 2;
      return;
    }
  } else {
    for (int w = 1; w <= 8; ++w) consider(places * w / units, false);  // the most that w waves hold
    consider(most, false);
  }
  if (p.cl > 1) {
    p.chunk = 1 << 30;
    p.nch = 1;
    return;
  }
  int64_t chunk = best == 1 ? max_keys : (keys + best - 1) / best;
  chunk = (chunk + 31) / 32 * 32;
  p.chunk = (int)std::min<int64_t>(chunk, 1 << 30);
  p.nch = (int)((max_keys + p.chunk - 1) / p.chunk);
}

Plan make_plan(const misa_problem_t* p, const misa_kv_cache_t* c, int Hq, int k,
               const misa_shared_prefix_t* share) {
  Plan pl;
  const int G = Hq / c->num_kv_heads;
  const int64_t T = p->num_queries, S = p->num_seqs, H = c->num_kv_heads;
  const bool grid = row_grid(p, c).rows > 0;
  auto tiles = [](int64_t rows, int64_t per) { return (rows + per - 1) / per; };
  if (k > 0) {
    pick_rows(pl.own, G, grid);
    const int64_t units = T * tiles(G, pl.own.rows) * H;
    split_keys(pl.own, units, k, k, !pl.own.tc, false);
    pl.own.bound = units * pl.own.nch;
  } else {
    const int64_t ng = share ? share->num_groups : 0, longest = ng ? share->max_len : 0;
    const int64_t per_seq = tiles(T, S) * G;
    pick_rows(pl.own, per_seq, grid);
    // what the prefixes hold is not read per sequence
    const int64_t keys = std::max<int64_t>(p->total_keys - S * longest, p->total_keys / 64) / S + 1;
    split_keys(pl.own, S * tiles(per_seq, pl.own.rows) * H, keys, p->max_seq_len,
               !pl.own.tc, !pl.own.tc);
    pl.own.bound = (T * G / pl.own.rows + S) * H * pl.own.nch;
    if (ng && longest > 0) {
      const int64_t per_group = tiles(T, ng) * G;
      pick_rows(pl.shared, per_group, grid);
      split_keys(pl.shared, ng * tiles(per_group, pl.shared.rows) * H, longest, longest, false, false);
      pl.shared.bound = (T * G / pl.shared.rows + ng) * H * pl.shared.nch;
    }
  }
  // The own launch joins the shared prefix's chunks itself where it has a row's own keys at hand.
  pl.finish = pl.shared.nch > 0 && pl.own.nch == 1 && !pl.own.tc;
  pl.nslots = (pl.finish ? 0 : pl.own.nch) + pl.shared.nch;
  pl.partial = pl.shared.nch > 0 || pl.own.nch > 1;
  pl.o_bytes = up256((size_t)(T * Hq) * pl.nslots * c->head_dim * 4);
  pl.lse_bytes = up256((size_t)(T * Hq) * pl.nslots * 4);
  return pl;
}

int check_attention(const misa_problem_t* p, const misa_kv_cache_t* c, int Hq,
                    const misa_shared_prefix_t* share) {
  int rc = check_batch(p);
  if (rc || (rc = check_cache(p, c, true))) return rc;
  if (Hq < 1 || Hq % c->num_kv_heads || Hq / c->num_kv_heads > 64) {
    set_error("num_q_heads %d must be a multiple of num_kv_heads %d, at most 64 times as many", Hq,
              c->num_kv_heads);
    return MISA_ERR_INVALID_ARG;
  }
  if ((int64_t)p->num_queries * Hq >= (int64_t(1) << 31) || p->max_seq_len > (1 << 30)) {
    set_error("attention: %d queries of %d heads, or max_seq_len %d, exceed the grid", p->num_queries, Hq,
              p->max_seq_len);
    return MISA_ERR_UNSUPPORTED;
  }
  if (share) {
    if (share->num_groups < 0 || share->max_len < 0 || share->max_len > p->max_seq_len) {
      set_error("shared prefixes need groups >= 0 and 0 <= max_len <= max_seq_len (groups=%d max_len=%d)",
                share->num_groups, share->max_len);
      return MISA_ERR_INVALID_ARG;
    }
    if (share->num_groups > 0 &&
        ((rc = check_ptr(share->seq_offsets, 4, "share seq_offsets")) || (rc = check_ptr(share->lens, 4, "share lens"))))
      return rc;
  }
  return MISA_OK;
}

int attend(const misa_problem_t* p, const misa_kv_cache_t* c, const void* q, int Hq,
           const misa_attention_opts_t* opts, const misa_shared_prefix_t* share, const int32_t* idx, int k,
           void* out, float* lse, void* ws, size_t ws_bytes, cudaStream_t st) {
  int rc;
  if (!opts) { set_error("options are NULL"); return MISA_ERR_INVALID_ARG; }
  if (!(opts->softcap >= 0.f) || !(fabsf(opts->scale) <= 3e38f) || !(opts->softcap <= 3e38f)) {
    set_error("scale must be finite and softcap finite and >= 0");
    return MISA_ERR_INVALID_ARG;
  }
  if (p->num_queries == 0) return MISA_OK;
  if ((rc = check_ptr(q, 16, "q")) || (rc = check_ptr(out, 16, "out")) || (rc = check_ptr(ws, 256, "workspace")))
    return rc;
  if ((lse && !aligned(lse, 4)) || (opts->slopes && !aligned(opts->slopes, 4))) {
    set_error("lse or slopes misaligned");
    return MISA_ERR_INVALID_ARG;
  }
  const Plan pl = make_plan(p, c, Hq, k, share);
  if (ws_bytes < pl.bytes()) {
    set_error("workspace too small: %zu < %zu", ws_bytes, pl.bytes());
    return MISA_ERR_WORKSPACE_TOO_SMALL;
  }
  if (q == out) { set_error("out must not be q: blocks read q after others have written"); return MISA_ERR_INVALID_ARG; }
  uint32_t* status = status_ptr();
  if (!status) { set_error("status word unavailable"); return MISA_ERR_CUDA; }
  AttendArgs a = {};
  a.c = cache_view(p, c);
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.qo = p->query_offsets;
  a.q_pos = p->q_pos;
  a.idx = idx;
  a.slopes = opts->slopes;
  a.status = status;
  const bool cap = opts->softcap > 0.f;
  // held finite, so that a product of 0 stays 0; a cap's rows then stay finite too
  auto finite = [](double x, double most) { return (float)std::max(-most, std::min(most, x)); };
  const double log2e = 1.4426950408889634, raw2 = opts->scale * log2e;
  a.raw2 = finite(raw2, FLT_MAX);
  a.scale2 = cap ? finite(2 * raw2 / opts->softcap, FLT_MAX) : a.raw2;
  if (cap) {
    a.cap2 = finite(opts->softcap * log2e, FLT_MAX / 4);
    a.inv_cap2 = finite(1 / (opts->softcap * log2e), FLT_MAX);
    a.series_max = finite(raw2 == 0 ? FLT_MAX : kSeries * opts->softcap * log2e / fabs(raw2), FLT_MAX);
  }
  const RowGrid grid = row_grid(p, c);
  if (grid.rows) {
    // a stride that nothing is multiplied by need not be a multiple of the unit
    a.unit = grid.unit;
    a.page_rows = (int)(c->page_stride / grid.unit);
    a.token_rows = (int)(c->token_stride / grid.unit);
    a.head_rows = (int)(c->head_stride / grid.unit);
    a.map_rows = (int)grid.rows;
    // Boxes of up to 64 consecutive rows of a page, at least the eight of a
    // swizzle pattern; where the tokens are packed they start anywhere.
    const int box = c->page_table ? std::gcd(c->page_size, 64) : 64;
    const bool apart = c->token_stride > 0 && (c->num_kv_heads == 1 || c->head_stride > 0) &&
                       (!c->page_table || c->num_pages <= 1 || c->page_stride > 0);
    a.box = box >= 8 && apart ? box : 0;
    a.box_align = a.box && c->page_table ? box : 1;
  }
  a.S = p->num_seqs;
  a.T = p->num_queries;
  a.Hq = Hq;
  a.Hkv = c->num_kv_heads;
  a.G = Hq / c->num_kv_heads;
  a.k = k;
  a.max_seq_len = p->max_seq_len;
  a.nslots = pl.nslots;
  a.cl = 1;
  a.most_cuts = a.most_steps = 1;
  if (share && pl.shared.nch) {
    a.ng = share->num_groups;
    a.max_shared = share->max_len;
    a.so = share->seq_offsets;
    a.slen = share->lens;
  }
  if (pl.partial) {
    a.part_o = static_cast<float*>(ws);
    a.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + pl.o_bytes);
  }
  if (pl.shared.nch) {
    AttendArgs b = a;
    b.chunk = pl.shared.chunk;
    b.nch_max = pl.shared.nch;
    b.slot0 = 0;
    if ((rc = launch_attend<kShared>(b, c->dtype, c->head_dim, pl.shared.tc, pl.shared.rows, pl.shared.bound, st))) return rc;
  }
  a.chunk = pl.own.chunk;
  a.nch_max = pl.own.nch;
  a.slot0 = pl.shared.nch;
  a.cl = pl.own.cl;
  a.finish = pl.finish;
  a.rows = pl.own.rows;
  if (pl.own.cuts) {
    a.blocks = num_sms() * 2;
    a.most_cuts = pl.own.cuts;
    a.most_steps = (p->max_seq_len + kStep - 1) / kStep;
    a.nch_max = 1 << 30;
  }
  a.shared_chunk = pl.shared.chunk;
  a.shared_nch = pl.shared.nch;
  if (pl.own.cl > 1 && !pl.finish) a.part_o = nullptr;
  rc = k > 0 ? launch_attend<kSelected>(a, c->dtype, c->head_dim, pl.own.tc, pl.own.rows, pl.own.bound, st)
             : launch_attend<kOwn>(a, c->dtype, c->head_dim, pl.own.tc, pl.own.rows, pl.own.bound, st);
  if (rc || !pl.partial || pl.finish) return rc;
  CombineArgs ca;
  ca.a = a;
  ca.own_chunk = pl.own.chunk;
  ca.own_max = pl.own.nch;
  ca.shared_chunk = pl.shared.chunk;
  ca.shared_max = pl.shared.nch;
  ca.own0 = pl.shared.nch;
  ca.selected = k > 0;
  return launch_combine(ca, c->dtype, c->head_dim, st);
}

}  // namespace
}  // namespace misa

using namespace misa;

extern "C" {

size_t misa_attention_workspace_size(const misa_problem_t* p, const misa_kv_cache_t* cache,
                                     int32_t num_q_heads, int32_t k, const misa_shared_prefix_t* share) {
  if (check_attention(p, cache, num_q_heads, share)) return 0;
  if (k < 0 || k > 65536 || (k > 0 && share)) {
    set_error("k=%d outside 0..65536, or shared prefixes with a selection", k);
    return 0;
  }
  return make_plan(p, cache, num_q_heads, k, share).bytes();
}

int misa_attention(const misa_problem_t* p, const misa_kv_cache_t* cache, const void* q, int32_t num_q_heads,
                   const misa_attention_opts_t* opts, const misa_shared_prefix_t* share, void* out, float* lse,
                   void* ws, size_t ws_bytes, misa_stream_t stream) {
  const int rc = check_attention(p, cache, num_q_heads, share);
  if (rc) return rc;
  return attend(p, cache, q, num_q_heads, opts, share, nullptr, 0, out, lse, ws, ws_bytes,
                static_cast<cudaStream_t>(stream));
}

int misa_attention_selected(const misa_problem_t* p, const misa_kv_cache_t* cache, const void* q,
                            int32_t num_q_heads, const misa_attention_opts_t* opts, const int32_t* idx, int32_t k,
                            void* out, float* lse, void* ws, size_t ws_bytes, misa_stream_t stream) {
  int rc = check_attention(p, cache, num_q_heads, nullptr);
  if (rc) return rc;
  if (k < 1 || k > 65536) { set_error("k=%d outside 1..65536", k); return MISA_ERR_INVALID_ARG; }
  if (p->num_queries > 0 && (rc = check_ptr(idx, 4, "idx"))) return rc;
  return attend(p, cache, q, num_q_heads, opts, nullptr, idx, k, out, lse, ws, ws_bytes,
                static_cast<cudaStream_t>(stream));
}

}  // extern "C"
