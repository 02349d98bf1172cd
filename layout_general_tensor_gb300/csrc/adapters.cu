// Low-rank adapters of many requests beside a shared projection
// (include/adapters.h).
//
// Bound: memory.  A row costs K + 2 N values and 2 rank (K + N) multiply-adds, a
// group its two matrices, so the whole adapter is one pass that keeps the first
// product's result u on the chip: no workspace, one launch.
//
// A tile is up to 8 NT rows of one group, done by a cluster of 1 to 8 CTAs:
//   u = x A^T:       every warp of the cluster takes a stretch of K for all of
//                    the tile's rows and the whole rank, m16n8k16 with the rank
//                    on the 16-side and rows on the 8-side (a single new token
//                    wastes the least so); the warps' sums are added through
//                    shared memory, the CTAs' through the cluster's, in order.
//   out = base + s u B^T: every warp takes blocks of 32 columns, rows on the
//                    16-side; u is in registers from here on.
// Fragments come straight from memory: the contraction may take its index in any
// order common to both operands, so a lane loads 16 (or 8) consecutive bytes of a
// row and uses them as the fragment's pairs.  Likewise the columns of a block of
// 32 are dealt to the instruction's 8-sides so that a lane ends up with eight
// neighbours of a row: base and out move in 16-byte pieces.
#include <algorithm>
#include <cstdint>

#include "adapters.h"
#include "groups.cuh"
#include "half_types.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace lgt {
namespace {

constexpr int kAdWarps = 8;
constexpr int kAdThreads = kAdWarps * 32;
constexpr int kAdMaxGroups = 1024;

struct AdapterArgs {
  const uint16_t *x, *a, *b, *base;
  uint16_t* out;
  const float* scales;
  const int32_t *offsets, *order;
  int64_t xs, bs, os;
  int32_t rows, groups, rank, n, k;
  uint32_t ctas;  // of a cluster
  int32_t copy;   // rows of no group go from base to out
};

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load16(const uint16_t* p, bool there) {
  return there ? *reinterpret_cast<const uint4*>(p) : make_uint4(0u, 0u, 0u, 0u);
}
__device__ __forceinline__ uint2 load8(const uint16_t* p, bool there) {
  return there ? *reinterpret_cast<const uint2*>(p) : make_uint2(0u, 0u);
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Two values as the sum of two pairs of the type.
template <bool BF16>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_pair16<BF16>(x, y);
  const float2 h = unpack_pair16<BF16>(hi);
  // (what is no number or infinite has nothing left over)
  lo = pack_pair16<BF16>(isfinite(h.x) ? x - h.x : 0.0f, isfinite(h.y) ? y - h.y : 0.0f);
}

template <int MT, int NT>
struct AdapterCfg {
  static constexpr int TOK = 8 * NT;                       // rows of a tile
  static constexpr int RANK = 16 * MT;                     // padded
  static constexpr int TOK16 = (TOK + 15) / 16 * 16;
  static constexpr int M2 = TOK16 / 16 == 1 || MT == 8 ? 1 : 2;  // 16-row groups of a warp in the second product
  static constexpr int SHARES = TOK16 / (16 * M2);         // warps that share a block of columns
  static constexpr int PITCH = RANK + 4;                   // fp32: 8 lanes' columns and 4 lanes' rows in 32 banks
  static constexpr int UPITCH = RANK + 8;                  // 16-bit
  static constexpr size_t PART = sizeof(float) * kAdWarps * TOK * PITCH;
  static constexpr size_t U = 2 * 2 * TOK16 * UPITCH;
  static size_t smem(int groups) { return PART + U + 4 * TOK16 * 2 + 4 * 32 + 8 * static_cast<size_t>(groups + 1); }
};

template <int MT, int NT, bool BF16>
__global__ void __launch_bounds__(kAdThreads, MT * NT <= 16 ? 2 : 1) adapters_kernel(const AdapterArgs a) {
  pdl_launch_dependents();
  using C = AdapterCfg<MT, NT>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  float* part = reinterpret_cast<float*>(smem_raw);
  uint16_t* uh = reinterpret_cast<uint16_t*>(smem_raw + C::PART);
  uint16_t* ul = uh + C::TOK16 * C::UPITCH;
  int32_t* row_of = reinterpret_cast<int32_t*>(smem_raw + C::PART + C::U);
  float* factor = reinterpret_cast<float*>(row_of + C::TOK16);
  uint32_t* scratch = reinterpret_cast<uint32_t*>(factor + C::TOK16);
  uint32_t* off = scratch + 32;
  uint32_t* first = off + a.groups + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l4 = lane >> 2, q = lane & 3;
  const uint32_t rank = a.ctas > 1 ? cluster_ctarank() : 0u;

  pdl_wait();
  group_rows<kAdThreads>(a.offsets, a.groups, a.rows, off, scratch);
  __syncthreads();
  group_tiles<kAdThreads>(a.groups, [&](uint32_t g) { return (off[g + 1] - off[g] + C::TOK - 1) / C::TOK; }, first, scratch + 16);
  __syncthreads();
  const uint32_t tiles = first[a.groups], clusters = gridDim.x / a.ctas;
  const int steps = (a.k + 31) / 32, blocks = (a.n + 31) / 32;

  for (uint32_t tile = blockIdx.x / a.ctas; tile < tiles; tile += clusters) {
    const uint32_t g = group_of(first, a.groups, tile);
    const uint32_t at = off[g] + (tile - first[g]) * C::TOK;
    const uint32_t count = min(static_cast<uint32_t>(C::TOK), off[g + 1] - at);
    if (threadIdx.x < C::TOK16) {
      int32_t r = -1;
      if (threadIdx.x < count) {
        r = static_cast<int32_t>(at + threadIdx.x);
        if (a.order) r = a.order[r];
        if (static_cast<uint32_t>(r) >= static_cast<uint32_t>(a.rows)) r = -1;
      }
      row_of[threadIdx.x] = r;
    }
    __syncthreads();

    // ------------------------------------------------------------ u = x A^T
    {
      float acc[MT][NT][4];
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.0f;
      const uint16_t* xr[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int32_t r = row_of[8 * j + l4];
        xr[j] = r >= 0 ? a.x + r * a.xs + q * 8 : nullptr;
      }
      const uint16_t* ar = a.a + (static_cast<int64_t>(g) * a.rank + l4) * a.k + q * 8;
      const int mine = static_cast<int>(rank) * kAdWarps + warp, all = static_cast<int>(a.ctas) * kAdWarps;
      const int s0 = static_cast<int>(static_cast<int64_t>(steps) * mine / all);
      const int s1 = static_cast<int>(static_cast<int64_t>(steps) * (mine + 1) / all);
#pragma unroll(MT * NT <= 2 ? 4 : MT * NT <= 8 ? 2 : 1)
      for (int s = s0; s < s1; ++s) {
        const int k = s * 32;
        const bool in = k + q * 8 < a.k;
        uint4 av[MT][2], xv[NT];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            av[i][h] = load16(ar + static_cast<int64_t>(16 * i + 8 * h) * a.k + k, in && 16 * i + 8 * h + l4 < a.rank);
#pragma unroll
        for (int j = 0; j < NT; ++j) xv[j] = load16(xr[j] + k, in && xr[j]);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            mma16816<BF16>(acc[i][j], av[i][0].x, av[i][1].x, av[i][0].y, av[i][1].y, xv[j].x, xv[j].y);
            mma16816<BF16>(acc[i][j], av[i][0].z, av[i][1].z, av[i][0].w, av[i][1].w, xv[j].z, xv[j].w);
          }
      }
      float* p = part + warp * C::TOK * C::PITCH;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            p[(8 * j + 2 * q + (e & 1)) * C::PITCH + 16 * i + l4 + 8 * (e >> 1)] = acc[i][j][e];
    }
    __syncthreads();
    constexpr int PER = C::RANK / 4;  // lanes of a row, a power of two
    float4 mine4[(C::TOK * PER + kAdThreads - 1) / kAdThreads];
#pragma unroll
    for (int it = 0; it < static_cast<int>(sizeof(mine4) / sizeof(float4)); ++it) {
      const int i = it * kAdThreads + threadIdx.x;
      float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (i < C::TOK * PER) {
        const int o = i / PER * C::PITCH + i % PER * 4;
#pragma unroll
        for (int w = 0; w < kAdWarps; ++w) {
          const float4 v = *reinterpret_cast<const float4*>(part + w * C::TOK * C::PITCH + o);
          s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        // (this thread alone reads and writes these places)
        if (a.ctas > 1) *reinterpret_cast<float4*>(part + o) = s;
      }
      mine4[it] = s;
    }
    if (a.ctas > 1) cluster_sync_all();
#pragma unroll
    for (int it = 0; it < static_cast<int>(sizeof(mine4) / sizeof(float4)); ++it) {
      const int i = it * kAdThreads + threadIdx.x;
      const int t = i / PER, c = i % PER * 4;
      const bool live = t < C::TOK;
      float4 s = mine4[it];
      if (a.ctas > 1 && live) {
        s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const uint32_t from = smem_u32(part + t * C::PITCH + c);
        for (uint32_t r = 0; r < a.ctas; ++r) {
          const float4 v = ld_cluster_f32x4(mapa_shared(from, r));
          s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
      }
      // (past the rank are sums of what x holds times 0, which is not 0 for an infinity)
      if (c >= a.rank) s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      // The row's power of two: its largest value goes to [0.5, 1).
      float most = fmaxf(fmaxf(fabsf(s.x), fabsf(s.y)), fmaxf(fabsf(s.z), fabsf(s.w)));
#pragma unroll
      for (int o = 1; o < PER; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      const int e = static_cast<int>(__float_as_uint(most) >> 23);  // (biased; no sign)
      const int p = e == 0 || e == 255 ? 0 : min(e - 126, 126);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - p) << 23);
      if (live) {
        uint32_t h0, h1, g0, g1;
        split_pair<BF16>(s.x * down, s.y * down, h0, g0);
        split_pair<BF16>(s.z * down, s.w * down, h1, g1);
        *reinterpret_cast<uint2*>(uh + t * C::UPITCH + c) = make_uint2(h0, h1);
        *reinterpret_cast<uint2*>(ul + t * C::UPITCH + c) = make_uint2(g0, g1);
        if (c == 0)
          factor[t] = __uint_as_float(static_cast<uint32_t>(127 + p) << 23) * (a.scales ? a.scales[g] : 1.0f);
      }
    }
    __syncthreads();

    // ------------------------------------------------------------ out = base + u B^T
    {
      constexpr int M2 = C::M2;
      const int share = warp % C::SHARES;
      uint2 hi[M2][MT][2], lo[M2][MT][2];
      int32_t row[M2][2];
      float f[M2][2];
#pragma unroll
      for (int m = 0; m < M2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int t = (share * M2 + m) * 16 + 8 * h + l4;
          const bool live = t < C::TOK;
          row[m][h] = live ? row_of[t] : -1;
          f[m][h] = live ? factor[t] : 0.0f;
#pragma unroll
          for (int s = 0; s < MT; ++s) {
            hi[m][s][h] = live ? *reinterpret_cast<const uint2*>(uh + t * C::UPITCH + 16 * s + 4 * q) : make_uint2(0u, 0u);
            lo[m][s][h] = live ? *reinterpret_cast<const uint2*>(ul + t * C::UPITCH + 16 * s + 4 * q) : make_uint2(0u, 0u);
          }
        }
      const int b0 = static_cast<int>(static_cast<int64_t>(blocks) * rank / a.ctas);
      const int b1 = static_cast<int>(static_cast<int64_t>(blocks) * (rank + 1) / a.ctas);
      const uint16_t* br = a.b + static_cast<int64_t>(g) * a.n * a.rank + 4 * q;
      for (int b = b0 + warp / C::SHARES; b < b1; b += kAdWarps / C::SHARES) {
        uint2 bv[4][MT];
        uint4 old[M2][2];
        const int n = b * 32;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = n + 8 * (l4 >> 1) + 2 * j + (l4 & 1);
#pragma unroll
          for (int s = 0; s < MT; ++s)
            bv[j][s] = load8(br + static_cast<int64_t>(c) * a.rank + 16 * s, c < a.n && 16 * s + 4 * q < a.rank);
        }
        const bool in = n + 8 * q < a.n;
#pragma unroll
        for (int m = 0; m < M2; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) old[m][h] = load16(a.base + row[m][h] * a.bs + n + 8 * q, in && row[m][h] >= 0);
#pragma unroll
        for (int m = 0; m < M2; ++m) {
          float acc[4][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
#pragma unroll
            for (int s = 0; s < MT; ++s) {
              mma16816<BF16>(acc[j], hi[m][s][0].x, hi[m][s][1].x, hi[m][s][0].y, hi[m][s][1].y, bv[j][s].x, bv[j][s].y);
              mma16816<BF16>(acc[j], lo[m][s][0].x, lo[m][s][1].x, lo[m][s][0].y, lo[m][s][1].y, bv[j][s].x, bv[j][s].y);
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t w[4] = {old[m][h].x, old[m][h].y, old[m][h].z, old[m][h].w};
            uint32_t y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 o = unpack_pair16<BF16>(w[j]);
              y[j] = pack_pair16<BF16>(fmaf(acc[j][2 * h], f[m][h], o.x), fmaf(acc[j][2 * h + 1], f[m][h], o.y));
            }
            if (in && row[m][h] >= 0) st_global_v4(a.out + row[m][h] * a.os + n + 8 * q, y[0], y[1], y[2], y[3]);
          }
        }
      }
    }
    // (the partial sums and the rows are used again: by this CTA's threads, and
    // the cluster's others have read them)
    if (a.ctas > 1)
      cluster_sync_all();
    else
      __syncthreads();
  }

  if (a.copy) {
    // Rows of no group: the places before the first group and behind the last.
    const uint32_t head = off[0], none = head + static_cast<uint32_t>(a.rows) - off[a.groups];
    const uint32_t pieces = static_cast<uint32_t>(a.n) / 8;
    for (uint32_t i = blockIdx.x; i < none; i += gridDim.x) {
      int32_t r = static_cast<int32_t>(i < head ? i : off[a.groups] + (i - head));
      if (a.order) r = a.order[r];
      if (static_cast<uint32_t>(r) >= static_cast<uint32_t>(a.rows)) continue;
      for (uint32_t c = threadIdx.x; c < pieces; c += kAdThreads)
        *reinterpret_cast<uint4*>(a.out + r * a.os + c * 8) = *reinterpret_cast<const uint4*>(a.base + r * a.bs + c * 8);
    }
  }
  if (a.ctas > 1) cluster_sync_all();
}

template <int MT, int NT, bool BF16>
cudaError_t launch_adapters_as(const AdapterArgs& a, unsigned clusters, cudaStream_t stream) {
  using C = AdapterCfg<MT, NT>;
  const cudaError_t e = set_smem_once<adapters_kernel<MT, NT, BF16>>(static_cast<int>(C::smem(kAdMaxGroups)));
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(adapters_kernel<MT, NT, BF16>, dim3(clusters * a.ctas), dim3(kAdThreads), C::smem(a.groups), stream,
                            a.ctas, a);
}

template <int MT, bool BF16>
cudaError_t launch_adapters_mt(const AdapterArgs& a, int nt, unsigned clusters, cudaStream_t stream) {
  return nt == 1 ? launch_adapters_as<MT, 1, BF16>(a, clusters, stream) : launch_adapters_as<MT, 4, BF16>(a, clusters, stream);
}

template <bool BF16>
cudaError_t launch_adapters(const AdapterArgs& a, int nt, unsigned clusters, cudaStream_t stream) {
  return a.rank <= 16   ? launch_adapters_mt<1, BF16>(a, nt, clusters, stream)
         : a.rank <= 32 ? launch_adapters_mt<2, BF16>(a, nt, clusters, stream)
         : a.rank <= 64 ? launch_adapters_mt<4, BF16>(a, nt, clusters, stream)
                        : launch_adapters_mt<8, BF16>(a, nt, clusters, stream);
}

}  // namespace
}  // namespace lgt

extern "C" gemm_status_t gemm_adapters_run(const gemm_adapters_desc_t* desc, const void* x, int64_t x_stride, const void* A,
                                           const void* B, const float* scales, const int32_t* offsets, const int32_t* order,
                                           int64_t rows, const void* base, int64_t base_stride, void* out,
                                           int64_t out_stride, void* stream) {
  using namespace lgt;
  if (!desc || rows < 0) return GEMM_ERR_INVALID_ARG;
  const gemm_adapters_desc_t& d = *desc;
  auto size = [](int64_t v) { return v >= 8 && v % 8 == 0 && v < (int64_t{1} << 30); };
  if (d.groups < 1 || d.groups > kAdMaxGroups || d.rank < 8 || d.rank > 128 || d.rank % 8 != 0 || !size(d.N) || !size(d.K) ||
      (d.dtype != GEMM_F16 && d.dtype != GEMM_BF16))
    return GEMM_ERR_INVALID_ARG;
  if (x_stride == 0) x_stride = d.K;
  if (base_stride == 0) base_stride = d.N;
  if (out_stride == 0) out_stride = d.N;
  for (int64_t v : {x_stride, base_stride, out_stride})
    if (v < 0 || v % 8 != 0 || v > (int64_t{1} << 32)) return GEMM_ERR_INVALID_ARG;
  if (x_stride < d.K || base_stride < d.N || out_stride < d.N || (out == base && out_stride != base_stride))
    return GEMM_ERR_INVALID_ARG;
  if (rows == 0) return GEMM_OK;
  if (!x || !A || !B || !offsets || !base || !out) return GEMM_ERR_INVALID_ARG;
  for (const void* p : {x, A, B, base, static_cast<const void*>(out)})
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return GEMM_ERR_ALIGNMENT;
  for (const void* p : {static_cast<const void*>(scales), static_cast<const void*>(offsets), static_cast<const void*>(order)})
    if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return GEMM_ERR_ALIGNMENT;
  if (rows > (int64_t{1} << 30)) return GEMM_ERR_UNSUPPORTED;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  AdapterArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.a = static_cast<const uint16_t*>(A);
  a.b = static_cast<const uint16_t*>(B);
  a.base = static_cast<const uint16_t*>(base);
  a.out = static_cast<uint16_t*>(out);
  a.scales = scales;
  a.offsets = offsets;
  a.order = order;
  a.xs = x_stride;
  a.bs = base_stride;
  a.os = out_stride;
  a.rows = static_cast<int32_t>(rows);
  a.groups = d.groups;
  a.rank = d.rank;
  a.n = static_cast<int32_t>(d.N);
  a.k = static_cast<int32_t>(d.K);
  a.copy = out != base;
  const int64_t busy = std::min<int64_t>(d.groups, rows);
  const int nt = rows > 8 * busy ? 4 : 1;
  const int64_t tiles = rows / (8 * nt) + busy;
  // A cluster as large as leaves a CTA for every SM, or what there is to share.
  a.ctas = 1;
  while (a.ctas < 8 && tiles * a.ctas * 2 <= sms && std::max(d.N, d.K) >= static_cast<int64_t>(a.ctas) * 512) a.ctas *= 2;
  const unsigned clusters = static_cast<unsigned>(std::min<int64_t>(tiles, 2 * sms / a.ctas));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = d.dtype == GEMM_BF16 ? launch_adapters<true>(a, nt, clusters, s) : launch_adapters<false>(a, nt, clusters, s);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  return GEMM_OK;
}
