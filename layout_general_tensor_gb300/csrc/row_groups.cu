// Rows put in order by group (include/row_groups.h): a stable counting sort.
//
// Bound: latency.  A row costs 12 bytes (131072 rows: 0.2 us of memory), so what
// counts is the number of dependent steps: one launch, the CTAs of one cluster
// with their counts in shared memory, no pass through global memory between (512
// rows of 128 groups 3.4 us).
//
// The rows are cut into equal runs, in order, one a warp, with a counter of its
// own for each group.  The first pass counts; then the counters become places (the
// groups before, the CTAs before, the warps before).  The second pass goes through
// the run 32 rows at a time; the lanes whose rows have the same group set their
// bits in one word of it, and a row's place is what the counter holds plus the bits
// below its own.  (Found by the match instruction instead, 131072 rows of 128
// groups took 33 us on 8 CTAs; by a vote on each bit of the number, with twice the
// warps, 9.8 us on 16 against 9.9, but 6.2 against 5.7 for 4096 rows.)
//
// A step of the second pass is some 40 wavefronts of shared memory, one of the first
// a fifth of that.  So where a warp has several steps, up to eight clusters do the
// whole first pass each, and each only its part of every run in the second: they need
// nothing of one another (131072 rows of 128 groups, one cluster 10.1 us, two 7.7,
// six 5.9; 4096 rows 6.0, eight 4.2).
#include <algorithm>
#include <cstdint>

#include "groups.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "row_groups.h"

namespace lgt {
namespace {

constexpr int kRgWarps = 16;
constexpr int kRgThreads = kRgWarps * 32;
constexpr int kRgMaxGroups = 1024;
constexpr unsigned kRgMaxCluster = 16;
constexpr uint32_t kRgBatch = 8;

struct RowGroupArgs {
  const int32_t* ids;
  int32_t *offsets, *order, *places;
  uint32_t rows, run;  // run: rows of a warp, a multiple of 32
  uint32_t lg_ctas;  // of a cluster
  uint32_t part;     // rows of a run that a cluster puts in place
  int32_t groups;
};

// A warp's word of a group: its lanes of the present step, its rows so far.
struct Bin {
  uint32_t lanes, count;
};

__device__ __forceinline__ uint32_t ld_shared_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ int32_t bin_of(const RowGroupArgs& a, int32_t id) {
  return id >= 0 && id < a.groups ? id : a.groups;
}

// 8 steps of a warp's rows, on their way at once (a step takes less than a trip to memory).
__device__ __forceinline__ void load_batch(const RowGroupArgs& a, uint32_t first, uint32_t i, uint32_t end, int32_t (&id)[kRgBatch]) {
#pragma unroll
  for (uint32_t j = 0; j < kRgBatch; ++j) {
    const uint32_t r = i + 32 * j + (threadIdx.x & 31);
    id[j] = r < end ? a.ids[first + r] : -1;
  }
}

// PARTS: several clusters (one does not pay for them: 512 rows 3.1 us, 3.4).
template <bool PARTS>
__global__ void __launch_bounds__(kRgThreads, 1) row_groups_kernel(const RowGroupArgs a) {
  pdl_launch_dependents();
  extern __shared__ __align__(8) uint8_t rg_smem[];
  __shared__ uint32_t total[kRgMaxGroups + 1];  // this CTA's rows of each group, read by the cluster's others
  __shared__ uint32_t all[kRgMaxGroups + 1], before[kRgMaxGroups + 1], first_of[kRgMaxGroups + 2];
  __shared__ uint32_t scratch[16];
  const int bins = a.groups + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank(), ctas = 1u << a.lg_ctas;
  Bin* bin = reinterpret_cast<Bin*>(rg_smem);  // [warp][bins]
  Bin* mine = bin + warp * bins;
  for (int i = lane; i < bins; i += 32) mine[i] = Bin{0u, 0u};
  __syncwarp();
  pdl_wait();
  const uint32_t first = (rank * kRgWarps + warp) * a.run;
  const uint32_t end = first < a.rows ? min(a.run, a.rows - first) : 0u;
  // this cluster's part of the run
  const uint32_t from = PARTS ? (blockIdx.x >> a.lg_ctas) * a.part : 0u, to = PARTS ? min(end, from + a.part) : end;
  int32_t id[kRgBatch];
  for (uint32_t i = 0; i < end; i += 32 * kRgBatch) {
    load_batch(a, first, i, end, id);
#pragma unroll
    for (uint32_t j = 0; j < kRgBatch; ++j)
      if (i + 32 * j + lane < end) {
        Bin* at = mine + bin_of(a, id[j]);
        atomicAdd(PARTS && i + 32 * j < from ? &at->lanes : &at->count, 1u);
      }
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kRgThreads) {
    uint32_t s = 0;
#pragma unroll
    for (int w = 0; w < kRgWarps; ++w) s += bin[w * bins + b].count + (PARTS ? bin[w * bins + b].lanes : 0u);
    total[b] = s;
  }
  cluster_sync_all();
  // Each group's rows in all CTAs and in those before this one.
  for (int b = threadIdx.x; b < bins; b += kRgThreads) {
    const uint32_t at = smem_u32(&total[b]);
    uint32_t sum = 0, low = 0;
#pragma unroll
    for (uint32_t c = 0; c < kRgMaxCluster; ++c) {
      const uint32_t n = c < ctas ? ld_shared_cluster_u32(mapa_shared(at, c)) : 0u;
      sum += n;
      low += c < rank ? n : 0u;
    }
    all[b] = sum;
    before[b] = low;
  }
  __syncthreads();
  group_tiles<kRgThreads>(bins, [&](uint32_t b) { return all[b]; }, first_of, scratch);
  __syncthreads();
  // The warps' counters become the places of their first rows.
  for (int b = threadIdx.x; b < bins; b += kRgThreads) {
    if (blockIdx.x == 0) a.offsets[b] = static_cast<int32_t>(first_of[b]);
    uint32_t at = first_of[b] + before[b];
    Bin n[kRgWarps];
#pragma unroll
    for (int w = 0; w < kRgWarps; ++w) n[w] = Bin{PARTS ? bin[w * bins + b].lanes : 0u, bin[w * bins + b].count};
#pragma unroll
    for (int w = 0; w < kRgWarps; ++w) {
      bin[w * bins + b].count = at + n[w].lanes;
      if (PARTS) bin[w * bins + b].lanes = 0u;
      at += n[w].lanes + n[w].count;
    }
  }
  cluster_sync_all();  // (the totals have been read; a CTA leaves its shared memory to no one before)
  const uint32_t below = (1u << lane) - 1u;
  const bool again = a.run > 32 * kRgBatch;  // (else they are still here)
  for (uint32_t i = again ? from : 0u; i < to; i += 32 * kRgBatch) {
    if (again) load_batch(a, first, i, to, id);
#pragma unroll
    for (uint32_t j = 0; j < kRgBatch; ++j) {
      if (i + 32 * j < from) continue;
      if (i + 32 * j >= to) break;
      const uint32_t r = i + 32 * j + lane;
      const bool live = r < to;
      Bin* at = mine + bin_of(a, id[j]);
      if (live) atomicOr(&at->lanes, 1u << lane);
      __syncwarp();
      const Bin now = *at;
      __syncwarp();
      const uint32_t rank_here = __popc(now.lanes & below);
      if (live && rank_here == 0) *at = Bin{0u, now.count + __popc(now.lanes)};
      __syncwarp();
      if (live) {
        const uint32_t place = now.count + rank_here;
        a.order[place] = static_cast<int32_t>(first + r);
        if (a.places) a.places[first + r] = static_cast<int32_t>(place);
      }
    }
  }
}

template <bool PARTS>
cudaError_t launch_row_groups(const RowGroupArgs& a, unsigned ctas, unsigned clusters, size_t smem, cudaStream_t stream) {
  constexpr auto kernel = row_groups_kernel<PARTS>;
  cudaError_t e = set_smem_once<kernel>(kRgWarps * (kRgMaxGroups + 1) * static_cast<int>(sizeof(Bin)));
  if (e == cudaSuccess && ctas > 8) e = allow_large_clusters_once<kernel>();
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(kernel, dim3(ctas * clusters), dim3(kRgThreads), smem, stream, ctas, a);
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
  // as many CTAs as keep every warp at eight steps or fewer, up to a cluster's most
  a.lg_ctas = 0;
  while (1u << a.lg_ctas < kRgMaxCluster && rows > (int64_t{kRgThreads} * 8 << a.lg_ctas)) ++a.lg_ctas;
  const unsigned ctas = 1u << a.lg_ctas;
  const int64_t warps = static_cast<int64_t>(ctas) * kRgWarps;
  a.run = static_cast<uint32_t>((rows + warps * 32 - 1) / (warps * 32) * 32);
  // (a GPU's SM groups hold six clusters of 16 at once with room to spare; one that has
  // to wait for another takes as long again: eight 10.5 us for 131072 rows, six 5.9)
  const uint32_t steps = a.run / 32, most = ctas > 8 ? 6 : 8, part = std::max(1u, (steps + most - 1) / most);
  const unsigned clusters = std::max(1u, (steps + part - 1) / part);
  a.part = part * 32;
  const int smem = kRgWarps * (groups + 1) * static_cast<int>(sizeof(Bin));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = clusters > 1 ? launch_row_groups<true>(a, ctas, clusters, static_cast<size_t>(smem), st)
                                     : launch_row_groups<false>(a, ctas, clusters, static_cast<size_t>(smem), st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  return GEMM_OK;
}
