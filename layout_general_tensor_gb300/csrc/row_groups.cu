// Rows put in order by group (include/row_groups.h): a stable counting sort.
//
// Bound: latency.  A row costs 12 bytes (131072 rows: 0.2 us of memory), so what
// counts is the number of dependent steps: one launch, the CTAs of one cluster
// with their counts in shared memory, no pass through global memory between.
//
// The rows are cut into equal runs, in order, one a warp, with a counter of its
// own for each group.  The first pass counts; then the counters become places (the
// groups before, the CTAs before, the warps before).  The second pass goes through
// the run 32 rows at a time; the lanes whose rows have the same group find each
// other by a vote on each bit of the number, and a row's place is what the counter
// holds plus the lanes of its group below it.  (The match instruction in the
// place of the votes, in both passes: 33 us for 131072 rows of 128 groups on 8
// CTAs, against VOTES.)
#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"
#include "row_groups.h"

namespace lgt {
namespace {

constexpr int kRgWarps = 32;
constexpr int kRgThreads = kRgWarps * 32;
constexpr int kRgMaxGroups = 1024;
constexpr unsigned kRgMaxCluster = 16;

struct RowGroupArgs {
  const int32_t* ids;
  int32_t *offsets, *order, *places;
  uint32_t rows, run;  // run: rows of a warp, a multiple of 32
  int32_t groups;
  int32_t bits;  // of a number up to `groups`
};

__device__ __forceinline__ uint32_t ld_shared_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ int32_t bin_of(const RowGroupArgs& a, int32_t id) {
  return id >= 0 && id < a.groups ? id : a.groups;
}

// A warp's rows from `first` on: how many each group has.
__device__ __forceinline__ void count_run(const RowGroupArgs& a, uint32_t first, uint32_t end, uint32_t* count) {
  const uint32_t lane = threadIdx.x & 31;
#pragma unroll 4
  for (uint32_t i = lane; i < end; i += 32) atomicAdd(&count[bin_of(a, a.ids[first + i])], 1u);
}

// And their places; `count` holds the place of each group's next row.
__device__ __forceinline__ void place_run(const RowGroupArgs& a, uint32_t first, uint32_t end, uint32_t* count) {
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t below = (1u << lane) - 1u;
  // (ids are asked for one step ahead)
  int32_t next = lane < end ? a.ids[first + lane] : -1;
#pragma unroll 1
  for (uint32_t i = 0; i < end; i += 32) {
    const uint32_t row = first + i + lane;
    const bool live = i + lane < end;
    const int32_t bin = bin_of(a, next);
    next = i + 32 + lane < end ? a.ids[row + 32] : -1;
    uint32_t same = __ballot_sync(0xffffffffu, live);
    for (int b = 0; b < a.bits; ++b) {
      const uint32_t set = __ballot_sync(0xffffffffu, bin >> b & 1);
      same &= bin >> b & 1 ? set : ~set;
    }
    const uint32_t at = count[bin];
    __syncwarp();
    if (live && (same & below) == 0) count[bin] = at + __popc(same);
    if (live) {
      const uint32_t place = at + __popc(same & below);
      a.order[place] = static_cast<int32_t>(row);
      if (a.places) a.places[row] = static_cast<int32_t>(place);
    }
    __syncwarp();
  }
}

__global__ void __launch_bounds__(kRgThreads, 1) row_groups_kernel(const RowGroupArgs a) {
  pdl_launch_dependents();
  extern __shared__ uint32_t rg_smem[];
  __shared__ uint32_t total[kRgMaxGroups + 1];  // this CTA's rows of each group, read by the cluster's others
  __shared__ uint32_t scan[kRgWarps];
  const int bins = a.groups + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank(), ctas = gridDim.x;
  uint32_t* mine = rg_smem + warp * bins;
  for (int i = lane; i < bins; i += 32) mine[i] = 0;
  __syncwarp();
  pdl_wait();
  const uint32_t first = (rank * kRgWarps + warp) * a.run;
  const uint32_t end = first < a.rows ? min(a.run, a.rows - first) : 0u;
  count_run(a, first, end, mine);
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kRgThreads) {
    uint32_t s = 0;
#pragma unroll
    for (int w = 0; w < kRgWarps; ++w) s += rg_smem[w * bins + b];
    total[b] = s;
  }
  cluster_sync_all();
  // Every thread one group: its rows in all CTAs and in those before this one.
  const int g = threadIdx.x;
  uint32_t all = 0, before = 0;
  if (g < a.groups) {
    const uint32_t at = smem_u32(&total[g]);
#pragma unroll
    for (uint32_t c = 0; c < kRgMaxCluster; ++c) {
      const uint32_t n = c < ctas ? ld_shared_cluster_u32(mapa_shared(at, c)) : 0u;
      all += n;
      before += c < rank ? n : 0u;
    }
  }
  uint32_t upto = all;  // rows of the groups up to this one
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) scan[warp] = upto;
  __syncthreads();
  {
    uint32_t s = lane < warp ? scan[lane] : 0u;
    upto += __reduce_add_sync(0xffffffffu, s);
  }
  if (rank == 0 && g < a.groups) {
    a.offsets[g + 1] = static_cast<int32_t>(upto);
    if (g == 0) a.offsets[0] = 0;
  }
  // The warps' counters become the places of their first rows.
  auto spread = [&](int b, uint32_t at) {
    uint32_t n[kRgWarps];
#pragma unroll
    for (int w = 0; w < kRgWarps; ++w) n[w] = rg_smem[w * bins + b];
#pragma unroll
    for (int w = 0; w < kRgWarps; ++w) {
      rg_smem[w * bins + b] = at;
      at += n[w];
    }
  };
  if (g < a.groups) spread(g, upto - all + before);
  if (g == a.groups - 1) {
    // (the rows of no group come behind the last)
    const uint32_t at = smem_u32(&total[a.groups]);
    uint32_t n = upto;
#pragma unroll
    for (uint32_t c = 0; c < kRgMaxCluster; ++c) n += c < rank ? ld_shared_cluster_u32(mapa_shared(at, c)) : 0u;
    spread(a.groups, n);
  }
  cluster_sync_all();  // (the totals have been read; a CTA leaves its shared memory to no one before)
  place_run(a, first, end, mine);
}

bool overlaps(const void* p, int64_t np, const void* q, int64_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && np > 0 && nq > 0 && a < b + static_cast<uintptr_t>(nq) * 4 && b < a + static_cast<uintptr_t>(np) * 4;
}

}  // namespace
}  // namespace lgt

extern "C" gemm_status_t gemm_row_groups(const int32_t* ids, int64_t rows, int32_t groups, int32_t* offsets, int32_t* order,
                                         int32_t* places, void* stream) {
  using namespace lgt;
  if (rows < 0 || groups < 1 || groups > kRgMaxGroups || !offsets || (rows > 0 && (!ids || !order)))
    return GEMM_ERR_INVALID_ARG;
  if (rows > (int64_t{1} << 30)) return GEMM_ERR_UNSUPPORTED;
  for (const void* p : {static_cast<const void*>(ids), static_cast<const void*>(offsets), static_cast<const void*>(order),
                        static_cast<const void*>(places)})
    if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return GEMM_ERR_ALIGNMENT;
  const void* span[4] = {ids, order, places, offsets};
  const int64_t count[4] = {rows, rows, rows, groups + 1};
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < i; ++j)
      if (overlaps(span[i], count[i], span[j], count[j])) return GEMM_ERR_INVALID_ARG;
  RowGroupArgs a;
  a.ids = ids;
  a.offsets = offsets;
  a.order = order;
  a.places = places;
  a.rows = static_cast<uint32_t>(rows);
  a.groups = groups;
  a.bits = 0;
  while (groups >> a.bits) ++a.bits;
  // as many CTAs as keep every warp at four steps or fewer, up to a cluster's most
  unsigned ctas = 1;
  while (ctas < kRgMaxCluster && rows > static_cast<int64_t>(ctas) * kRgThreads * 4) ctas *= 2;
  const int64_t warps = static_cast<int64_t>(ctas) * kRgWarps;
  a.run = static_cast<uint32_t>((rows + warps * 32 - 1) / (warps * 32) * 32);
  const int smem = kRgWarps * (groups + 1) * 4;
  cudaError_t e = set_smem_once<row_groups_kernel>(kRgWarps * (kRgMaxGroups + 1) * 4);
  if (e == cudaSuccess && ctas > 8) e = cudaFuncSetAttribute(row_groups_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess)
    e = launch_pdl_cluster(row_groups_kernel, dim3(ctas), dim3(kRgThreads), static_cast<size_t>(smem),
                           static_cast<cudaStream_t>(stream), ctas, a);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  return GEMM_OK;
}
