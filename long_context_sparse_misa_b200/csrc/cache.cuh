// The key/value cache as the device sees it, shared by the append and the
// attention kernels: where a token's row is, and how a query row is found.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace misa {

struct CacheView {
  uint16_t* k;
  uint16_t* v;
  const int32_t* table;  // nullptr: packed
  const int64_t* ko;
  int64_t table_stride, page_stride, token_stride, head_stride, total_keys;
  int page_size, page_shift, num_pages, pages_per_seq;  // page_shift < 0: not a power of two
};

// Elements from the base to token `pos` (>= 0) of sequence `seq`, head 0, or
// -1 where the page table or the packed buffer has no such row.
__device__ __forceinline__ int64_t cache_row(const CacheView& c, int seq, int pos) {
  if (c.table) {
    const int pi = c.page_shift >= 0 ? pos >> c.page_shift : pos / c.page_size;
    if (pi >= c.pages_per_seq) return -1;
    const int pg = __ldg(c.table + seq * c.table_stride + pi);
    if (pg < 0 || pg >= c.num_pages) return -1;
    return pg * c.page_stride + (int64_t)(pos - pi * c.page_size) * c.token_stride;
  }
  const int64_t r = __ldg(c.ko + seq) + pos;
  return r >= 0 && r < c.total_keys ? r * c.token_stride : -1;
}

// The last s with off[s] <= x (off non-decreasing, n entries, off[0] <= x),
// found by a whole warp, 32 probes at a time: two rounds of loads for up to
// 1024 sequences where one lane's bisection takes ten.
__device__ __forceinline__ int warp_segment(const int32_t* __restrict__ off, int n, int x) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int i = lane * step;
    const unsigned hit = __ballot_sync(0xffffffffu, i < n && __ldg(off + lo + i) <= x);
    const int c = max(__popc(hit) - 1, 0) * step;
    lo += c;
    n = min(step, n - c);
  }
  return lo;
}

__device__ __forceinline__ float to_float(uint16_t b, __nv_bfloat16) { return bf16_bits_to_float(b); }
__device__ __forceinline__ float to_float(uint16_t b, __half) { return __half2float(__ushort_as_half(b)); }

// Two fp32 values rounded to the 16-bit type, the first in the low half.
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __nv_bfloat16) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __half) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// launch_pdl with clusters of `cluster` blocks along x (the grid is a multiple of it).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_cluster(void (*kern)(KArgs...), dim3 grid, dim3 block, int cluster, size_t smem,
                               cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Argument checks (cache.cu).
int check_batch(const misa_problem_t* p);
int check_cache(const misa_problem_t* p, const misa_kv_cache_t* c, bool need_v);
CacheView cache_view(const misa_problem_t* p, const misa_kv_cache_t* c);
// Tensor map (abi.cu) of `rows` rows of `dim` 16-bit elements, `stride` elements apart, for gathers of
// four rows of 64 elements.
int make_rows_map(CUtensorMap* map, const void* base, int64_t rows, int dim, int64_t stride, bool fp16);
// Tensor map (abi.cu) of the cache as [pages, heads, page, dim], boxes of `box` rows of 64 elements.
int make_box_map(CUtensorMap* map, const void* base, const CacheView& c, int heads, int dim, int box, bool fp16);

}  // namespace misa
