// Work over groups of rows whose sizes are on the device, shared by the kernels
// that take offsets (gemm_grouped.cu, adapters.cu).
#pragma once
#include <cstdint>

namespace lgt {

__device__ __forceinline__ uint32_t scan_max(uint32_t v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) >= o) v = max(v, y);
  }
  return v;
}
__device__ __forceinline__ uint32_t scan_add(uint32_t v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) >= o) v += y;
  }
  return v;
}

// By a whole CTA of THREADS threads: off[g], the groups' first rows, never
// decreasing and never past `rows`.  off holds groups + 1 values, scratch one for
// each warp.  A barrier of the CTA has to follow.
template <int THREADS>
__device__ __forceinline__ void group_rows(const int32_t* offsets, int32_t groups, int32_t rows, uint32_t* off,
                                           uint32_t* scratch) {
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t n = static_cast<uint32_t>(groups) + 1;
  const uint32_t per = (n + THREADS - 1) / THREADS;
  const uint32_t lo = min(tid * per, n), hi = min(lo + per, n);
  uint32_t most = 0;
  for (uint32_t i = lo; i < hi; ++i) {
    most = max(most, static_cast<uint32_t>(min(max(offsets[i], 0), rows)));
    off[i] = most;
  }
  const uint32_t upto = scan_max(most);
  if (lane == 31) scratch[warp] = upto;
  __syncthreads();
  uint32_t before = __shfl_up_sync(0xffffffffu, upto, 1);
  if (lane == 0) before = 0;
  for (uint32_t w = 0; w < warp; ++w) before = max(before, scratch[w]);
  for (uint32_t i = lo; i < hi; ++i) off[i] = max(off[i], before);
}

// Likewise first[i], the tiles before entry i, where entry i has tiles_of(i) of
// them; first[entries] is their number.
template <int THREADS, typename TilesOf>
__device__ __forceinline__ void group_tiles(int32_t entries, TilesOf tiles_of, uint32_t* first, uint32_t* scratch) {
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t n = static_cast<uint32_t>(entries) + 1;
  const uint32_t per = (n + THREADS - 1) / THREADS;
  const uint32_t lo = min(tid * per, n), hi = min(lo + per, n);
  uint32_t sum = 0;
  for (uint32_t i = lo; i < hi; ++i) {
    first[i] = sum;
    if (i + 1 < n) sum += tiles_of(i);
  }
  const uint32_t upto = scan_add(sum);
  if (lane == 31) scratch[warp] = upto;
  __syncthreads();
  uint32_t before = upto - sum;
  for (uint32_t w = 0; w < warp; ++w) before += scratch[w];
  for (uint32_t i = lo; i < hi; ++i) first[i] += before;
}

// The entry of a tile: the last one whose first tile is not past it (an entry
// without tiles has its successor's).
__device__ __forceinline__ uint32_t group_of(const uint32_t* first, int32_t groups, uint32_t tile) {
  uint32_t g = 0, n = static_cast<uint32_t>(groups);
  while (n > 1) {
    const uint32_t half = n >> 1;
    if (first[g + half] <= tile) g += half;
    n -= half;
  }
  return g;
}

}  // namespace lgt
