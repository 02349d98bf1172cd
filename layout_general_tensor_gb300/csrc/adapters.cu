// Low-rank adapters of many requests beside a shared projection
// (include/adapters.h).
//
// Bound: memory.  A row costs K + 2 N values and 2 rank (K + N) multiply-adds, a
// group its two matrices, so the whole adapter is one pass that keeps the first
// product's result u on the chip: no workspace, one launch.  Many rows come near
// that (16384 rows, K = N = 4096, rank 64: 76 us, 80 % of a copy's rate).  Few are a
// chain of trips to memory, one after the other: offsets, order, rows, the joins of
// u, results (one row 5.8 us, 60 rows of 60 adapters 8.1, 801 rows of 13 and 198 of
// none, 3000 x 2880, 10.5).
//
// For few rows (for many: adapters_tc_kernel below) a tile is up to 8 NT rows of one
// group, done by a cluster of 1 to 8 CTAs:
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
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <new>

#include "adapters.h"
#include "groups.cuh"
#include "half_types.cuh"
#include "kernels.h"
#include "plan.h"
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
// A lane's values of a row for the second product: eight of every 32, which are two
// steps of it, or four of 16 where that is the rank.
template <int MT>
struct RankPiece {
  static constexpr int COUNT = MT / 2, VALUES = 8, STEPS = 2;
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t* p, bool there) { v = load16(p, there); }
  __device__ __forceinline__ uint2 step(int s) const { return s ? make_uint2(v.z, v.w) : make_uint2(v.x, v.y); }
};
template <>
struct RankPiece<1> {
  static constexpr int COUNT = 1, VALUES = 4, STEPS = 1;
  uint2 v;
  __device__ __forceinline__ void load(const uint16_t* p, bool there) {
    v = there ? *reinterpret_cast<const uint2*>(p) : make_uint2(0u, 0u);
  }
  __device__ __forceinline__ uint2 step(int) const { return v; }
};

// A value's size where it has one.  (A row's power of two goes by its finite values: with
// an infinity's, the others could pass fp16's largest and be infinite too.)
__device__ __forceinline__ float finite_size(float x) {
  const float size = fabsf(x);
  return size < INFINITY ? size : 0.0f;
}

// 2^n for n from -149 to 127.
__device__ __forceinline__ float power_of_two(int n) { return __uint_as_float(n >= -126 ? static_cast<uint32_t>(127 + n) << 23 : 1u << (n + 149)); }

// The power of two that takes a row's largest value to [0.5, 1), for bf16 to [2^-9, 2^-8)
// so that no sum over the rank with bf16 weights passes fp32's range, and what the second
// product of a row is multiplied with: the scale over that power.  Where this would pass
// fp32's range, though with small or large weights the result does not, u takes as much
// of it as is beyond; fp16's u, which has no room above, leaves the largest number (what
// is not 0 then has a result that fp16 does not hold).
template <bool BF16>
__device__ __forceinline__ float2 row_power(float most, float scale) {
  const int e = max(static_cast<int>(__float_as_uint(most) >> 23), 1);  // (biased; no sign)
  int n = (BF16 ? 118 : 126) - e;
  const uint32_t size = __float_as_uint(scale) & 0x7fffffffu;
  const bool some = size != 0 && size < 0x7f800000u;
  const int s = size >> 23 ? static_cast<int>(size >> 23) - 126 : -117 - __clz(size);  // |scale| is in [2^(s - 1), 2^s)
  if (some) n = min(BF16 ? max(n, s - 128) : n, s + 125);  // (|factor| in [2^-126, 2^128), u below 2^128)
  const int once = min(-n, 126);
  float factor = scale * power_of_two(once) * power_of_two(-n - once);
  if (!BF16 && some) factor = fminf(fmaxf(factor, -FLT_MAX), FLT_MAX);
  return make_float2(power_of_two(n), factor);
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack_pair16_rz(float lo, float hi) {
  uint32_t w;
  if constexpr (BF16)
    asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  else
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
  return w;
}

// The lesser of two pairs, one that is no number if either is.
template <bool BF16>
__device__ __forceinline__ uint32_t min_pair16(uint32_t a, uint32_t b) {
  uint32_t w;
  if constexpr (BF16)
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(w) : "r"(a), "r"(b));
  else
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(w) : "r"(a), "r"(b));
  return w;
}

// Values times the row's power of two, as the sum of two of the type each, in pairs.
// The parts of a value that is not 0 have its sign and are not 0 either, so that an
// infinite weight gives an infinity and not the difference of two, or 0 times one: what
// is left of a value cut towards 0, or two halves of one that the type holds (the least
// steps of the type are rounded to it, twice 2^-24 for fp16).
// (Nearly all values are of the first kind, which the least of what is left shows: above
// the type's least step for every one of them.  Without `there`, for rows and columns that
// the tile does not have, zeros stay zeros: else the second kind would be the rule, 16384
// rows, rank 128, 83.8 us against 81.6.)
template <bool BF16>
__device__ __forceinline__ float2 two_parts(float x, float h, float l, float half) {
  constexpr float kLeast = BF16 ? 0x1p-133f : 0x1p-24f;
  if (!isfinite(h)) return make_float2(h, h);
  if (l == 0.0f) {
    l = h - half;
    h = half;
  }
  return h == 0.0f && x != 0.0f ? make_float2(copysignf(kLeast, x), copysignf(kLeast, x)) : make_float2(h, l);
}
template <bool BF16, int PAIRS>
__device__ __forceinline__ void split_pairs(const float (&x)[2 * PAIRS], float power, bool there, uint32_t (&hi)[PAIRS], uint32_t (&lo)[PAIRS]) {
  uint32_t least = BF16 ? 0x7f7f7f7fu : 0x7bff7bffu;
#pragma unroll
  for (int i = 0; i < PAIRS; ++i) {
    const float v0 = x[2 * i] * power, v1 = x[2 * i + 1] * power;
    hi[i] = pack_pair16_rz<BF16>(v0, v1);
    const float2 cut = unpack_pair16<BF16>(hi[i]);
    lo[i] = pack_pair16<BF16>(v0 - cut.x, v1 - cut.y);
    least = min_pair16<BF16>(least, lo[i] & 0x7fff7fffu);
  }
  const float2 all = unpack_pair16<BF16>(least);
  constexpr float kLeast = BF16 ? 0x1p-133f : 0x1p-24f;
  if (!there || (all.x > kLeast && all.y > kLeast)) return;
#pragma unroll
  for (int i = 0; i < PAIRS; ++i) {
    const float2 cut = unpack_pair16<BF16>(hi[i]), left = unpack_pair16<BF16>(lo[i]);
    const float2 half = unpack_pair16<BF16>(pack_pair16_rz<BF16>(cut.x * 0.5f, cut.y * 0.5f));
    const float2 a = two_parts<BF16>(x[2 * i], cut.x, left.x, half.x), b = two_parts<BF16>(x[2 * i + 1], cut.y, left.y, half.y);
    hi[i] = pack_pair16<BF16>(a.x, b.x);
    lo[i] = pack_pair16<BF16>(a.y, b.y);
  }
}

// Rows of no group, at the places before the first group and behind the last, go
// from base to out, as tiles of their own behind the groups': `tile` of `per` rows,
// a row a warp, of which this is number `warp` of `warps` (of a cluster's).
__device__ __forceinline__ uint32_t other_rows(const AdapterArgs& a, const uint32_t* off) {
  return a.copy ? off[0] + static_cast<uint32_t>(a.rows) - off[a.groups] : 0u;
}
__device__ __forceinline__ void copy_others(const AdapterArgs& a, const uint32_t* off, uint32_t tile, uint32_t per, uint32_t warp,
                                            uint32_t warps) {
  const uint32_t from = tile * per, rows = min(per, other_rows(a, off) - from), pieces = static_cast<uint32_t>(a.n) / 8;
  for (uint32_t i = warp; i < rows; i += warps) {
    const uint32_t place = from + i;
    int32_t r = static_cast<int32_t>(place < off[0] ? place : off[a.groups] + (place - off[0]));
    if (a.order) r = a.order[r];
    if (static_cast<uint32_t>(r) >= static_cast<uint32_t>(a.rows)) continue;
    const uint16_t* src = a.base + r * a.bs;
    uint16_t* dst = a.out + r * a.os;
    for (uint32_t c = threadIdx.x & 31; c < pieces; c += 8 * 32) {  // (eight on their way at once)
      uint4 v[8];
#pragma unroll
      for (uint32_t j = 0; j < 8; ++j) v[j] = load16(src + static_cast<int64_t>(c + 32 * j) * 8, c + 32 * j < pieces);
#pragma unroll
      for (uint32_t j = 0; j < 8; ++j)
        if (c + 32 * j < pieces) *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(c + 32 * j) * 8) = v[j];
    }
  }
}

template <int MT, int NT>
struct AdapterCfg {
  static constexpr int TOK = 8 * NT;                       // rows of a tile
  static constexpr int RANK = 16 * MT;                     // padded
  static constexpr int TOK16 = (TOK + 15) / 16 * 16;
  static constexpr int M2 = TOK16 / 16 == 1 || MT == 8 ? 1 : 2;  // 16-row groups of a warp in the second product
  static constexpr int SHARES = TOK16 / (16 * M2);         // warps that share a block of columns
  static constexpr int BATCH = MT * M2 == 1 ? 4 : MT * M2 <= 4 ? 2 : 1;  // blocks of columns on their way, as registers allow
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
  const uint32_t all_tiles = tiles + (other_rows(a, off) + C::TOK - 1) / C::TOK;
  const int steps = (a.k + 31) / 32, blocks = (a.n + 31) / 32;

  for (uint32_t tile = blockIdx.x / a.ctas; tile < all_tiles; tile += clusters) {
    if (tile >= tiles) {
      copy_others(a, off, tile - tiles, C::TOK, rank * kAdWarps + warp, a.ctas * kAdWarps);
      continue;
    }
    const uint32_t g = group_of(first, a.groups, tile);
    const uint32_t at = off[g] + (tile - first[g]) * C::TOK;
    const uint32_t count = min(static_cast<uint32_t>(C::TOK), off[g + 1] - at);
    const float scale = a.scales ? a.scales[g] : 1.0f;
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
    // What the second product reads, a batch of blocks of 32 columns at a time; the
    // first batch is on its way while the sums are joined.
    const int share = warp % C::SHARES, apart = kAdWarps / C::SHARES;
    const int b0 = static_cast<int>(static_cast<int64_t>(blocks) * rank / a.ctas) + warp / C::SHARES;
    const int b1 = static_cast<int>(static_cast<int64_t>(blocks) * (rank + 1) / a.ctas);
    using Piece = RankPiece<MT>;
    const uint16_t* br = a.b + static_cast<int64_t>(g) * a.n * a.rank + Piece::VALUES * q;
    Piece bv[C::BATCH][4][Piece::COUNT];
    uint4 old[C::BATCH][C::M2][2];
    int32_t row[C::M2][2];
#pragma unroll
    for (int m = 0; m < C::M2; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = (share * C::M2 + m) * 16 + 8 * h + l4;
        row[m][h] = t < C::TOK ? row_of[t] : -1;
      }
    auto load_blocks = [&](int b) {
#pragma unroll
      for (int i = 0; i < C::BATCH; ++i) {
        const bool in = b + i * apart < b1;
        const int n = (b + i * apart) * 32;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = n + 8 * (l4 >> 1) + 2 * j + (l4 & 1);
#pragma unroll
          for (int s = 0; s < Piece::COUNT; ++s)
            bv[i][j][s].load(br + static_cast<int64_t>(c) * a.rank + 4 * Piece::VALUES * s,
                             in && c < a.n && Piece::VALUES * (4 * s + q) < a.rank);
        }
#pragma unroll
        for (int m = 0; m < C::M2; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            old[i][m][h] = load16(a.base + row[m][h] * a.bs + n + 8 * q, in && n + 8 * q < a.n && row[m][h] >= 0);
      }
    };
    load_blocks(b0);
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
      float most = fmaxf(fmaxf(finite_size(s.x), finite_size(s.y)), fmaxf(finite_size(s.z), finite_size(s.w)));
#pragma unroll
      for (int o = 1; o < PER; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      const float2 power = row_power<BF16>(most, scale);
      if (live) {
        uint32_t hi[2], lo[2];
        split_pairs<BF16, 2>({s.x, s.y, s.z, s.w}, power.x, c < a.rank && t < static_cast<int>(count), hi, lo);
        *reinterpret_cast<uint2*>(uh + t * C::UPITCH + c) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2*>(ul + t * C::UPITCH + c) = make_uint2(lo[0], lo[1]);
        if (c == 0) factor[t] = power.y;
      }
    }
    __syncthreads();

    // ------------------------------------------------------------ out = base + u B^T
    {
      constexpr int M2 = C::M2;
      Piece hi[M2][Piece::COUNT][2], lo[M2][Piece::COUNT][2];
      float f[M2][2];
#pragma unroll
      for (int m = 0; m < M2; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int t = (share * M2 + m) * 16 + 8 * h + l4;
          const bool live = t < C::TOK;
          f[m][h] = live ? factor[t] : 0.0f;
#pragma unroll
          for (int s = 0; s < Piece::COUNT; ++s) {
            hi[m][s][h].load(uh + t * C::UPITCH + Piece::VALUES * (4 * s + q), live);
            lo[m][s][h].load(ul + t * C::UPITCH + Piece::VALUES * (4 * s + q), live);
          }
        }
      for (int b = b0; b < b1; b += C::BATCH * apart) {
        if (b > b0) load_blocks(b);
#pragma unroll
        for (int i = 0; i < C::BATCH; ++i) {
          const int n = (b + i * apart) * 32 + 8 * q;
          const bool in = b + i * apart < b1 && n < a.n;
#pragma unroll
          for (int m = 0; m < M2; ++m) {
            float acc[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
#pragma unroll
              for (int s = 0; s < Piece::COUNT; ++s)
#pragma unroll
                for (int k = 0; k < Piece::STEPS; ++k) {
                  const uint2 b2 = bv[i][j][s].step(k), h0 = hi[m][s][0].step(k), h1 = hi[m][s][1].step(k);
                  const uint2 l0 = lo[m][s][0].step(k), l1 = lo[m][s][1].step(k);
                  mma16816<BF16>(acc[j], h0.x, h1.x, h0.y, h1.y, b2.x, b2.y);
                  mma16816<BF16>(acc[j], l0.x, l1.x, l0.y, l1.y, b2.x, b2.y);
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t w[4] = {old[i][m][h].x, old[i][m][h].y, old[i][m][h].z, old[i][m][h].w};
              uint32_t y[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 o = unpack_pair16<BF16>(w[j]);
                y[j] = pack_pair16<BF16>(fmaf(acc[j][2 * h], f[m][h], o.x), fmaf(acc[j][2 * h + 1], f[m][h], o.y));
              }
              if (in && row[m][h] >= 0) st_global_v4(a.out + row[m][h] * a.os + n, y[0], y[1], y[2], y[3]);
            }
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

  if (a.ctas > 1) cluster_sync_all();
}

// ------------------------------------------------------------ many rows
//
// The same pass on tcgen05: a tile is up to 128 rows of one group, done by a
// cluster of 1 to 8 CTAs (an SM moves some 60 bytes a ns, and where there are
// fewer tiles than SMs that is the limit), each with a stretch of K, then one of N:
//   u = x A^T:    rows on the instruction's M side (lanes of tensor memory), rank
//                 on its N side; x and A come by a ring of copies, x's rows by
//                 their numbers, four a copy, where there is an order.
// The CTAs leave their parts of u in shared memory, and each adds all of them, in
// order, and keeps the sum's two parts of 16 bits.  Then
//   out^T = B u^T: columns of out on the M side, 128 at a time, rows on the N
//                 side in steps of 16; sixteen warps add base, whose pieces are on
//                 their way a block ahead, through shared memory, where a transposing
//                 load and store of 8 x 8 pieces turn them to the accumulator's
//                 order and back.
//
// Roles (672 threads): warps 0..3 copies of x (0: of A too, 1: of B), warp 4
// tensor memory and products, warps 5..20 results.  (A thread issues a copy of
// four rows in 44 ns: with two such warps 96 us for 16384 rows in an order, rank
// 16, against 79.)
constexpr int kAtcThreads = 672;
constexpr int kAtcMmaWarp = 4, kAtcEpiWarp0 = 5, kAtcEpiWarps = 16;
constexpr uint32_t kAtcRows = 128;
constexpr uint32_t kAtcTile = 128 * 128;               // 128 rows of 64 values
constexpr uint32_t kAtcMaxStages = 8;
constexpr uint32_t kAtcPieces = 2;                     // of base, a warp (three: 32768 rows 147 to 151 us, K = 64 51 to 49)
constexpr uint32_t kAtcStaging = kAtcEpiWarps * kAtcPieces * 2048;
constexpr uint32_t kAtcBars = 2 * kAtcMaxStages + 16;  // (15, and what follows is loaded 16 bytes at a time)
static_assert(kAtcBars * 8 % 16 == 0);
constexpr uint32_t kAtcSmem = 227 * 1024;
constexpr uint64_t kAtcSettleNs = 200ull * 1000ull * 1000ull;

struct AdapterTcArgs {
  CUtensorMap tm_x, tm_a, tm_b;
  AdapterArgs p;
  DeviceStatus* status;
  uint64_t wait_limit_ns;
  uint32_t rank16, chunks;  // the rank in steps of 16; in stretches of 64
  uint32_t height;  // a tile's rows at most, a multiple of 16
  uint32_t stages, stage_bytes;
  uint32_t region, parts;  // bytes of the ring, and then of u, B and this CTA's part of u, which begins at `parts`
  uint32_t idesc_u, idesc_out;  // the second without N
  int32_t withhold;
};

// SHARED: clusters of several CTAs.
template <bool BF16, bool SHARED>
__global__ void __launch_bounds__(kAtcThreads, 1) adapters_tc_kernel(const __grid_constant__ AdapterTcArgs t) {
  pdl_launch_dependents();
  const AdapterArgs& a = t.p;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw_base);
  const uint32_t u_hi = base, u_lo = base + t.chunks * kAtcTile, b_ring = base + 2 * t.chunks * kAtcTile;
  const uint32_t parts = base + t.parts;
  const uint32_t staging = base + t.region;
  const uint32_t bar0 = staging + kAtcStaging;
  uint8_t* rest = smem + t.region + kAtcStaging + kAtcBars * 8;
  int32_t* row_of = reinterpret_cast<int32_t*>(rest);                 // [2][128], of this tile and the next
  float* factor = reinterpret_cast<float*>(rest + 1024);              // [128]
  volatile uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(rest + 1536);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(rest + 1540);
  uint32_t* scratch = reinterpret_cast<uint32_t*>(rest + 1544);       // [2][32]
  uint32_t* off = scratch + 64;
  uint32_t* first = off + a.groups + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = SHARED ? cluster_ctarank() : 0u;
  const uint32_t ctas = SHARED ? a.ctas : 1u;
  auto full = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty = [&](uint32_t s) { return bar0 + 8u * (kAtcMaxStages + s); };
  auto rows_full = [&](uint32_t b) { return bar0 + 8u * (2 * kAtcMaxStages + b); };
  const uint32_t u_done = bar0 + 8u * (2 * kAtcMaxStages + 2), u_full = u_done + 8, tile_done = u_done + 16, end_bar = u_done + 24;
  auto b_full = [&](uint32_t b) { return bar0 + 8u * (2 * kAtcMaxStages + 6 + b); };
  auto out_full = [&](uint32_t b) { return bar0 + 8u * (2 * kAtcMaxStages + 8 + b); };
  auto out_empty = [&](uint32_t b) { return bar0 + 8u * (2 * kAtcMaxStages + 10 + b); };
  const uint32_t results_done = bar0 + 8u * (2 * kAtcMaxStages + 12), parts_full = results_done + 8, parts_read = results_done + 16;
  auto given_up = [&](bool got) {
    if (!got) {
      *abort_flag = 1;
      t.status->where = warp;
      t.status->code = GEMM_ERR_TIMEOUT;
    }
    return got;
  };
  auto wait = [&](uint32_t bar, uint32_t parity) { return given_up(mbar_wait_bounded(bar, parity, t.wait_limit_ns, abort_flag)); };
  auto warp_wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)); };
  // (what the cluster's other CTAs complete)
  auto wait_cluster = [&](uint32_t bar, uint32_t parity) {
    return given_up(mbar_wait_bounded_cluster(bar, parity, t.wait_limit_ns, abort_flag));
  };
  auto arrive_all = [&](uint32_t bar) {  // in every CTA, once a warp
    __syncwarp();
    if (lane < static_cast<int>(ctas)) mbar_arrive_cluster(mapa_shared(bar, static_cast<uint32_t>(lane)));
  };

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < t.stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(u_done, 1);     // this CTA's part of the first product is
    mbar_init(u_full, SHARED ? kAtcEpiWarps : 4);  // u's 16-bit parts are in shared memory
    mbar_init(tile_done, 1);  // u and B have been read
    mbar_init(results_done, kAtcEpiWarps);
    mbar_init(parts_full, kAtcEpiWarps * ctas);  // every CTA's part is in its shared memory
    mbar_init(parts_read, kAtcEpiWarps * ctas);  // this CTA's part has been read
    mbar_init(end_bar, 1);
    for (uint32_t b = 0; b < 2; ++b) {
      mbar_init(rows_full(b), kAtcMmaWarp);
      mbar_init(b_full(b), 1);
      mbar_init(out_full(b), 1);
      mbar_init(out_empty(b), kAtcEpiWarps);
    }
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&t.tm_x);
    tma_prefetch_desc(&t.tm_a);
    tma_prefetch_desc(&t.tm_b);
  }
  if (warp == kAtcMmaWarp) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), 512);
    tmem_relinquish();
  }
  pdl_wait();
  group_rows<kAtcThreads>(a.offsets, a.groups, a.rows, off, scratch);
  __syncthreads();
  group_tiles<kAtcThreads>(a.groups, [&](uint32_t g) { return (off[g + 1] - off[g] + t.height - 1) / t.height; }, first, scratch + 32);
  tc_fence_before();
  __syncthreads();
  if constexpr (SHARED) cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tiles = first[a.groups], turn0 = blockIdx.x / ctas, turns = gridDim.x / ctas;
  // This CTA's blocks of K and of N.
  const int nkb = (a.k + TILE_K - 1) / TILE_K, nnb = (a.n + 127) / 128;
  const int kb0 = static_cast<int>(static_cast<int64_t>(nkb) * rank / ctas), kb1 = static_cast<int>(static_cast<int64_t>(nkb) * (rank + 1) / ctas);
  const int nb0 = static_cast<int>(static_cast<int64_t>(nnb) * rank / ctas), nb1 = static_cast<int>(static_cast<int64_t>(nnb) * (rank + 1) / ctas);
  // A tile: its group, first place and rows.
  struct Tile {
    uint32_t g, at, count;
  };
  auto tile_at = [&](uint32_t i) {
    Tile w;
    w.g = group_of(first, a.groups, i);
    const uint32_t len = off[w.g + 1] - off[w.g], n = (len + t.height - 1) / t.height;
    const uint32_t width = ((len + n - 1) / n + 15) & ~15u;
    w.at = off[w.g] + (i - first[w.g]) * width;
    w.count = min(width, off[w.g + 1] - w.at);
    return w;
  };
  const uint32_t u_tmem = tmem, out_tmem = tmem + 128;

  if (warp < kAtcMmaWarp) {
    // ------------------------------------------------------------ copies
    uint32_t s = 0, phase = 0, it = 0, issued = 0, b_uses = 0;
    bool ok = true;
    for (uint32_t i = turn0; ok && i < tiles; i += turns, ++it) {
      const Tile w = tile_at(i);
      int32_t* rows = row_of + (it & 1) * kAtcRows;
      // u, B and the parts of the tile before lie where the ring is.  (And the
      // results of the one before that, whose rows stood here, were done before its
      // u was made.)
      if (it > 0 && !(ok = warp_wait(tile_done, (it - 1) & 1u) && (!SHARED || __all_sync(0xffffffffu, wait_cluster(parts_read, (it - 1) & 1u))))) break;
      fence_proxy_async_smem();
      int32_t r = -1;
      const uint32_t place = warp * 32 + lane;
      if (place < w.count) {
        r = static_cast<int32_t>(w.at + place);
        if (a.order) r = a.order[r];
        if (static_cast<uint32_t>(r) >= static_cast<uint32_t>(a.rows)) r = -1;
      }
      rows[place] = r;
      __syncwarp();
      if (lane == 0) mbar_arrive(rows_full(it & 1));
      if (!(ok = warp_wait(rows_full(it & 1), it >> 1 & 1u))) break;
      // (by fours as far as the tile has rows, or all of a box)
      const uint32_t fours = (w.count + 3) / 4, load_bytes = (a.order ? fours * 512 : t.height * 128) + t.rank16 * 16 * 128;
      // A warp without copies passes a tile's stages over: nothing would bind it to the
      // others, and it could miss that a stage was used twice.  (All stages are empty
      // when a tile begins.)
      const bool copies = a.order ? static_cast<uint32_t>(warp) < fours || warp == 0 : warp == 0;
      if (!copies) {
        const uint32_t to = s + static_cast<uint32_t>(kb1 - kb0);
        phase ^= to / t.stages & 1u;
        s = to % t.stages;
      }
      if (elect_one()) {
        for (int kb = kb0; copies && kb < kb1; ++kb) {
          if (!(ok = wait(empty(s), phase ^ 1u))) break;
          const uint32_t dst = base + s * t.stage_bytes;
          if (warp == 0) {
            mbar_arrive_expect_tx(full(s), load_bytes);
            if (!(t.withhold && blockIdx.x == 0 && issued == 0))
              tma_load_3d(dst + kAtcTile, &t.tm_a, full(s), kb * TILE_K, 0, static_cast<int32_t>(w.g));
          }
          if (a.order) {
#pragma unroll 4
            for (uint32_t j = warp; j < fours; j += kAtcMmaWarp) {
              int4 r = *reinterpret_cast<const int4*>(rows + 4 * j);
              // (a row past the last gives zeros)
              r.x = r.x < 0 ? a.rows : r.x;
              r.y = r.y < 0 ? a.rows : r.y;
              r.z = r.z < 0 ? a.rows : r.z;
              r.w = r.w < 0 ? a.rows : r.w;
              tma_gather4(dst + j * 512, &t.tm_x, full(s), kb * TILE_K, r);
            }
          } else if (warp == 0) {
            tma_load_2d(dst, &t.tm_x, full(s), kb * TILE_K, static_cast<int32_t>(w.at));
          }
          ++issued;
          if (++s == t.stages) {
            s = 0;
            phase ^= 1u;
          }
        }
        // B's blocks, from when the ring is done with and, where the parts lie in
        // their place, those have been read
        if (warp == 1 && ok && (ok = wait(u_done, it & 1u) && (!SHARED || t.parts > 2 * t.chunks * kAtcTile || wait_cluster(parts_read, it & 1u)))) {
          fence_proxy_async_smem();
          for (int b = nb0; b < nb1; ++b, ++b_uses) {
            // (what the products of the block before the last have read is free once they are done)
            if (b_uses >= 2 && !(ok = wait(out_full(b_uses & 1u), (b_uses >> 1 & 1u) ^ 1u))) break;
            mbar_arrive_expect_tx(b_full(b_uses & 1u), t.chunks * kAtcTile);
            for (uint32_t c = 0; c < t.chunks; ++c)
              tma_load_3d(b_ring + ((b_uses & 1u) * t.chunks + c) * kAtcTile, &t.tm_b, b_full(b_uses & 1u),
                          static_cast<int32_t>(64 * c), b * 128, static_cast<int32_t>(w.g));
          }
        }
      }
      ok = __all_sync(0xffffffffu, ok);
    }
  } else if (warp == kAtcMmaWarp) {
    // ------------------------------------------------------------ products
    if (elect_one()) {
      const uint64_t x_desc = sw128_desc(base, 16u, 1024u), a_desc = sw128_desc(base + kAtcTile, 16u, 1024u);
      const uint64_t hi_desc = sw128_desc(u_hi, 16u, 1024u), lo_desc = sw128_desc(u_lo, 16u, 1024u);
      const uint64_t b_desc = sw128_desc(b_ring, 16u, 1024u);
      uint32_t s = 0, phase = 0, it = 0, uses = 0;
      bool ok = true;
      for (uint32_t i = turn0; ok && i < tiles; i += turns, ++it) {
        const Tile w = tile_at(i);
        // (u of the tile before has been read: its parts were full)
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!(ok = wait(full(s), phase))) break;
          tc_fence_after();
          const uint64_t xd = x_desc + s * (t.stage_bytes >> 4), ad = a_desc + s * (t.stage_bytes >> 4);
#pragma unroll
          for (int k = 0; k < TILE_K / 16; ++k)
            tc_mma_f16_ss(u_tmem, xd + 2 * k, ad + 2 * k, t.idesc_u, kb > kb0 || k > 0 ? 1u : 0u);
          tc_commit(empty(s));
          if (++s == t.stages) {
            s = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        tc_commit(u_done);
        if (!(ok = wait(u_full, it & 1u))) break;
        const uint32_t idesc = t.idesc_out | ((w.count + 15) & ~15u) >> 3 << 17;
        for (int b = nb0; b < nb1; ++b, ++uses) {
          const uint32_t buf = uses & 1u;
          if (!(ok = wait(b_full(buf), uses >> 1 & 1u) && wait(out_empty(buf), (uses >> 1 & 1u) ^ 1u))) break;
          tc_fence_after();
          const uint32_t d = out_tmem + buf * 128;
          for (uint32_t k = 0; k < t.rank16; ++k) {
            const uint32_t at = (k >> 2) * (kAtcTile >> 4) + (k & 3) * 2;
            const uint64_t bd = b_desc + buf * t.chunks * (kAtcTile >> 4) + at;
            tc_mma_f16_ss(d, bd, hi_desc + at, idesc, k > 0 ? 1u : 0u);
            tc_mma_f16_ss(d, bd, lo_desc + at, idesc, 1u);
          }
          tc_commit(out_full(buf));
        }
        if (!ok) break;
        tc_commit(tile_done);
      }
      tc_commit(end_bar);
    }
  } else {
    // ------------------------------------------------------------ results
    const uint32_t quad = static_cast<uint32_t>(warp & 3), share = static_cast<uint32_t>(warp - kAtcEpiWarp0) / 4;
    const uint32_t mine = staging + static_cast<uint32_t>(warp - kAtcEpiWarp0) * kAtcPieces * 2048u;
    const uint32_t row8 = static_cast<uint32_t>(lane >> 2), piece = static_cast<uint32_t>(lane & 3);
    // places in a piece of 32 rows of 64 bytes, as in the grouped products' results
    const uint32_t put = (lane & 7u) * 64u + ((static_cast<uint32_t>(lane >> 3) ^ (lane >> 1 & 3u)) << 4);
    const uint32_t get = row8 * 64u + ((piece ^ (row8 >> 1 & 3u)) << 4);
    // A part of u: rows of 16 rank16 values, whose 16-byte pieces are exchanged by
    // the row's number within eight, or four where they are no multiple of eight.  A
    // warp writes a quarter of its 32 rows, a thread adds one
    // of a row.
    const uint32_t turn = t.rank16 % 2 == 0 ? 7u : 3u, pitch = t.rank16 * 64u;
    const uint32_t put_row = quad * 32u + lane, add_row = static_cast<uint32_t>(threadIdx.x - kAtcEpiWarp0 * 32) >> 2;
    uint32_t it = 0, uses = 0;
    bool ok = true;
    for (uint32_t i = turn0; ok && i < tiles; i += turns, ++it) {
      const Tile w = tile_at(i);
      if (!(ok = warp_wait(rows_full(it & 1), it >> 1 & 1u))) break;
      const int32_t* rows = row_of + (it & 1) * kAtcRows;
      const float scale = a.scales ? a.scales[w.g] : 1.0f;
      // The four warps of a quarter of the lanes share the rows, 32 each, or, where
      // there are fewer, the blocks of columns.
      const uint32_t by_rows = w.count > 64 ? 4u : w.count > 32 ? 2u : 1u, every = 4u / by_rows;
      const uint32_t tok0 = share % by_rows * 32u;
      const int skip = static_cast<int>(share / by_rows);
      // Pieces of base: 32 rows of 32 columns, of each block of 128.
      const int n0 = static_cast<int>(quad * 32 + piece * 8);
      int32_t r[4];
#pragma unroll
      for (uint32_t j = 0; j < 4; ++j) r[j] = rows[tok0 + 8 * j + row8];
      uint32_t fetched = 0, used = 0;
      int ahead = nb0 + skip;
      auto fetch = [&]() {
        const int n = ahead * 128 + n0;
        if (ahead < nb1 && n < a.n) {
          const uint32_t dst = mine + (fetched % kAtcPieces) * 2048u + get;
#pragma unroll
          for (uint32_t j = 0; j < 4; ++j)
            if (r[j] >= 0) cp_async_16(dst + j * 512u, a.base + r[j] * a.bs + n);
        }
        cp_async_commit();
        ++fetched;
        ahead += static_cast<int>(every);
      };
      for (uint32_t b = 0; b + 1 < kAtcPieces; ++b) fetch();
      // (The rows' factors of the tile before are in use until its results are done.)
      if (SHARED || share == 0)
        if (!(ok = warp_wait(u_done, it & 1u) && (it == 0 || warp_wait(results_done, (it - 1) & 1u)))) break;
      if constexpr (SHARED) {
        // This CTA's part.
        tc_fence_after();
        {
          uint32_t v[32];
          const uint32_t c0 = share * t.rank16;  // in pieces of 4
  #pragma unroll
          for (uint32_t k = 0; k < 8; ++k)
            if (k < t.rank16) tc_ld_32x32b_x4(u_tmem + (quad * 32u << 16) + 4 * (c0 + k), v + 4 * k);
          tc_wait_ld_regs(v);
  #pragma unroll
          for (uint32_t k = 0; k < 8; ++k)
            if (k < t.rank16)
              st_shared_v4(parts + put_row * pitch + (((c0 + k) ^ (put_row & turn)) << 4), v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        }
        tc_fence_before();
        arrive_all(parts_full);
        if (!(ok = __all_sync(0xffffffffu, wait_cluster(parts_full, it & 1u)))) break;
        // The sum of all parts; its row's power of two, which takes the largest value to [0.5, 1); its two parts of 16 bits.
        {
          float4 v[8];
  #pragma unroll
          for (uint32_t k = 0; k < 8; ++k) v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          // (every fourth piece of a row, so that four lanes read 64 bytes together)
          for (uint32_t from = 0; from < ctas; ++from) {
            const uint32_t local = parts + add_row * pitch, at = mapa_shared(local, from);
  #pragma unroll
            for (uint32_t k = 0; k < 8; ++k)
              if (k < t.rank16) {
                const uint32_t o = ((piece + 4 * k) ^ (add_row & turn)) << 4;
                const float4 x = from == rank ? ld_shared_f32x4(local + o) : ld_cluster_f32x4(at + o);
                v[k].x += x.x, v[k].y += x.y, v[k].z += x.z, v[k].w += x.w;
              }
          }
          float most = 0.0f;
  #pragma unroll
          for (uint32_t k = 0; k < 8; ++k) {
            // (past the rank are sums of what x holds times 0, which is not 0 for an infinity)
            if (k >= t.rank16 || static_cast<int>(4 * (piece + 4 * k)) >= a.rank) v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            most = fmaxf(most, fmaxf(fmaxf(finite_size(v[k].x), finite_size(v[k].y)), fmaxf(finite_size(v[k].z), finite_size(v[k].w))));
          }
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
          const float2 power = row_power<BF16>(most, scale);
  #pragma unroll
          for (uint32_t k = 0; k < 8; ++k)
            if (k < t.rank16) {
              uint32_t hi[2], lo[2];
              split_pairs<BF16, 2>({v[k].x, v[k].y, v[k].z, v[k].w}, power.x, static_cast<int>(4 * (piece + 4 * k)) < a.rank && add_row < w.count, hi, lo);
              const uint32_t c = 4 * (piece + 4 * k);
              const uint32_t to = (c >> 6) * kAtcTile + add_row * 128 + (((c & 63u) >> 3) ^ (add_row & 7u)) * 16 + (c & 4u) * 2;
              st_shared_v2(u_hi + to, hi[0], hi[1]);
              st_shared_v2(u_lo + to, lo[0], lo[1]);
            }
          if (piece == 0) factor[add_row] = power.y;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(u_full);
        // (behind the stores, which have taken what was read: an arrival alone does not
        // wait for loads)
        arrive_all(parts_read);
      } else if (share == 0) {
        // u, a row a lane: the power of two that takes its largest value to [0.5, 1), then its two parts of 16 bits.
        tc_fence_after();
        const uint32_t row = quad * 32 + lane, from = u_tmem + (quad * 32u << 16);
        float most = 0.0f;
        for (uint32_t c = 0; c < t.rank16 * 16; c += 16) {
          uint32_t v[16];
          tc_ld_32x32b_x16(from + c, v);
          tc_wait_ld_regs(v);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (static_cast<int>(c) + e < a.rank) most = fmaxf(most, finite_size(__uint_as_float(v[e])));
        }
        const float2 power = row_power<BF16>(most, scale);
        for (uint32_t c = 0; c < t.rank16 * 16; c += 16) {
          uint32_t v[16];
          tc_ld_32x32b_x16(from + c, v);
          tc_wait_ld_regs(v);
          const uint32_t at = (c >> 6) * kAtcTile + row * 128;
#pragma unroll
          for (uint32_t j = 0; j < 2; ++j) {
            // (past the rank are sums of what x holds times 0, which is not 0 for an infinity)
            const bool in = c + 8 * j < static_cast<uint32_t>(a.rank);
            float x[8];
#pragma unroll
            for (uint32_t e = 0; e < 8; ++e) x[e] = in ? __uint_as_float(v[8 * j + e]) : 0.0f;
            uint32_t hi[4], lo[4];
            split_pairs<BF16, 4>(x, power.x, in && row < w.count, hi, lo);
            const uint32_t to = at + ((((c & 63u) >> 3) + j) ^ (row & 7u)) * 16;
            st_shared_v4(u_hi + to, hi[0], hi[1], hi[2], hi[3]);
            st_shared_v4(u_lo + to, lo[0], lo[1], lo[2], lo[3]);
          }
        }
        factor[row] = power.y;
        tc_fence_before();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(u_full);
      }
      if (!(ok = warp_wait(u_full, it & 1u))) break;
      float2 f[4];  // of rows 8 e + 2 piece and the next
#pragma unroll
      for (uint32_t e = 0; e < 4; ++e) f[e] = *reinterpret_cast<const float2*>(factor + tok0 + 8 * e + 2 * piece);
      for (int b = nb0; ok && b < nb1; ++b, ++uses) {
        const uint32_t buf = uses & 1u;
        const bool turn_here = static_cast<uint32_t>(b - nb0) % every == static_cast<uint32_t>(skip);
        if (turn_here) fetch();
        if (!(ok = warp_wait(out_full(buf), uses >> 1 & 1u))) break;
        tc_fence_after();
        // (the sums are free as soon as they have been read, before the results are stored)
        auto done = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(out_empty(buf));
        };
        if (turn_here) {
          const uint32_t here = mine + (used++ % kAtcPieces) * 2048u;
          const int n = b * 128 + n0;
          if (tok0 < w.count) {
            uint32_t x[16], y[16];
            tc_ld_16x256b_x4(out_tmem + buf * 128 + tok0 + (quad * 32u << 16), x);
            tc_ld_16x256b_x4(out_tmem + buf * 128 + tok0 + ((quad * 32u + 16u) << 16), y);
            cp_async_wait<kAtcPieces - 1>();
            __syncwarp();
            tc_wait_ld_regs(x);
            tc_regs_after_wait(y);
            done();
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e) {
              const uint4 old = ldmatrix_x4_trans(here + put + e * 512u);
              auto sum = [&](uint32_t lo, uint32_t hi, uint32_t o) {
                const float2 was = unpack_pair16<BF16>(o);
                return pack_pair16<BF16>(fmaf(__uint_as_float(lo), f[e].x, was.x), fmaf(__uint_as_float(hi), f[e].y, was.y));
              };
              stmatrix_x4_trans(here + put + e * 512u, sum(x[4 * e], x[4 * e + 1], old.x), sum(x[4 * e + 2], x[4 * e + 3], old.y),
                                sum(y[4 * e], y[4 * e + 1], old.z), sum(y[4 * e + 2], y[4 * e + 3], old.w));
            }
            __syncwarp();
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e) {
              const uint4 v = ld_shared_v4(here + get + e * 512u);
              if (r[e] >= 0 && n < a.n) st_global_v4(a.out + r[e] * a.os + n, v.x, v.y, v.z, v.w);
            }
          } else {
            done();
          }
        } else {
          done();
        }
      }
      if (lane == 0) mbar_arrive(results_done);
    }
    cp_async_wait<0>();
    // (the tiles of rows of no group go on where this cluster's turns leave off)
    const uint32_t all_tiles = tiles + (other_rows(a, off) + kAtcRows - 1) / kAtcRows;
    for (uint32_t i = turn0 + it * turns; ok && i < all_tiles; i += turns)
      copy_others(a, off, i - tiles, kAtcRows, rank * kAtcEpiWarps + (warp - kAtcEpiWarp0), ctas * kAtcEpiWarps);
  }

  // ------------------------------------------------------------ end
  __syncthreads();
  if (*abort_flag) {
    // Copies that were made may still be landing, on a barrier that will not
    // complete: they take microseconds, and are given far more.
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < kAtcSettleNs) {
    }
  }
  if (warp == kAtcMmaWarp) {
    volatile int no_abort = 0;
    mbar_wait_bounded(end_bar, 0, drain_ns(t.wait_limit_ns), &no_abort);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (SHARED) cluster_sync_all();  // (nobody's parts or barriers are in use any more)
  tc_fence_after();
  if (warp == kAtcMmaWarp) tmem_dealloc(tmem, 512);
}

template <int MT, int NT, bool BF16>
cudaError_t launch_adapters_as(const AdapterArgs& a, unsigned clusters, cudaStream_t stream) {
  using C = AdapterCfg<MT, NT>;
  const cudaError_t e = set_smem_once<adapters_kernel<MT, NT, BF16>>(static_cast<int>(C::smem(kAdMaxGroups)));
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(adapters_kernel<MT, NT, BF16>, dim3(clusters * a.ctas), dim3(kAdThreads), C::smem(a.groups), stream,
                            a.ctas, a);
}

// (nt: as gemm_adapters_run chooses them)
template <int MT, bool BF16>
cudaError_t launch_adapters_mt(const AdapterArgs& a, int nt, unsigned clusters, cudaStream_t stream) {
  if (nt == 1) return launch_adapters_as<MT, 1, BF16>(a, clusters, stream);
  if constexpr (MT <= 4)
    if (nt == 2) return launch_adapters_as<MT, 2, BF16>(a, clusters, stream);
  if constexpr (MT != 4)
    if (nt == 4) return launch_adapters_as<MT, 4, BF16>(a, clusters, stream);
  return cudaErrorInvalidValue;
}

template <bool BF16>
cudaError_t launch_adapters(const AdapterArgs& a, int nt, unsigned clusters, cudaStream_t stream) {
  return a.rank <= 16   ? launch_adapters_mt<1, BF16>(a, nt, clusters, stream)
         : a.rank <= 32 ? launch_adapters_mt<2, BF16>(a, nt, clusters, stream)
         : a.rank <= 64 ? launch_adapters_mt<4, BF16>(a, nt, clusters, stream)
                        : launch_adapters_mt<8, BF16>(a, nt, clusters, stream);
}

// [d2][d1][d0], dense, by boxes of 64 x box1.
bool encode_dense(CUtensorMap* map, const void* ptr, bool bf16, int64_t d0, int64_t d1, int64_t d2, uint32_t box1) {
  auto enc = get_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d0), static_cast<cuuint64_t>(d1), static_cast<cuuint64_t>(d2)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d0) * 2, static_cast<cuuint64_t>(d0 * d1) * 2};
  cuuint32_t box[3] = {64, box1, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(ptr), dims,
             strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// x's rows, boxes of 64 values of box1 rows.
bool encode_x(CUtensorMap* map, const void* ptr, bool bf16, int64_t k, int64_t rows, int64_t stride, uint32_t box1) {
  auto enc = get_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride) * 2};
  cuuint32_t box[2] = {64, box1};
  cuuint32_t estr[2] = {1, 1};
  return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(ptr), dims,
             strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool BF16>
cudaError_t launch_adapters_tc(const AdapterTcArgs& t, unsigned clusters, cudaStream_t stream) {
  if (t.p.ctas == 1) {
    const cudaError_t e = set_smem_once<adapters_tc_kernel<BF16, false>>(static_cast<int>(kAtcSmem));
    if (e != cudaSuccess) return e;
    return launch_pdl(adapters_tc_kernel<BF16, false>, dim3(clusters), dim3(kAtcThreads), kAtcSmem, stream, t);
  }
  const cudaError_t e = set_smem_once<adapters_tc_kernel<BF16, true>>(static_cast<int>(kAtcSmem));
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(adapters_tc_kernel<BF16, true>, dim3(clusters * t.p.ctas), dim3(kAtcThreads), kAtcSmem, stream, t.p.ctas, t);
}

// Clusters of `ctas` that run at once; < 0: an error.
template <bool BF16>
int resident_adapter_clusters(unsigned ctas) {
  if (set_smem_once<adapters_tc_kernel<BF16, true>>(static_cast<int>(kAtcSmem)) != cudaSuccess) return -1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kAtcThreads);
  cfg.dynamicSmemBytes = kAtcSmem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {ctas, 1, 1};
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  return cudaOccupancyMaxActiveClusters(&n, adapters_tc_kernel<BF16, true>, &cfg) == cudaSuccess ? n : -1;
}

uint64_t adapters_wait_limit() {
  const char* s = std::getenv("LGT_GEMM_WAIT_LIMIT_MS");
  if (s && *s) {
    const double ms = std::atof(s);
    if (ms > 0) return static_cast<uint64_t>(ms * 1e6);
  }
  return 2000ull * 1000ull * 1000ull;  // 2 s
}

}  // namespace
}  // namespace lgt

struct gemm_adapters_plan {
  gemm_adapters_desc_t d;
  int device = -1;
  int sms = 0;
  int resident[4] = {0, 0, 0, 0};  // clusters of 1, 2, 4, 8 CTAs of the form for many rows that run at once
  int tile_rows = 0;  // LGT_GEMM_ADAPTERS_ROWS: rows of a tile of the form for few rows
  int form = -1;  // LGT_GEMM_ADAPTERS_FORM: 0 the first form, 1, 2, 4, 8 the one for many rows with that many CTAs a tile
  lgt::DeviceStatus* d_status = nullptr;
  uint64_t wait_limit_ns = 0;
  int withhold_armed = 0;  // gemm_adapters_withhold_load: the next run of the large form withholds a load (one shot)
};

extern "C" {

gemm_status_t gemm_adapters_create(const gemm_adapters_desc_t* desc, gemm_adapters_plan_t** plan) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  *plan = nullptr;
  if (!desc) return GEMM_ERR_INVALID_ARG;
  const gemm_adapters_desc_t& d = *desc;
  auto size = [](int64_t v) { return v >= 8 && v % 8 == 0 && v < (int64_t{1} << 30); };
  if (d.groups < 1 || d.groups > lgt::kAdMaxGroups || d.rank < 8 || d.rank > 128 || d.rank % 8 != 0 || !size(d.N) ||
      !size(d.K) || (d.dtype != GEMM_F16 && d.dtype != GEMM_BF16))
    return GEMM_ERR_INVALID_ARG;
  gemm_adapters_plan* p = new (std::nothrow) gemm_adapters_plan();
  if (!p) return GEMM_ERR_CUDA;
  p->d = d;
  p->wait_limit_ns = lgt::adapters_wait_limit();
  if (const char* rows = std::getenv("LGT_GEMM_ADAPTERS_ROWS"); rows && *rows) {
    p->tile_rows = std::atoi(rows);
    if ((d.rank > 64 && p->tile_rows == 16) || (d.rank > 32 && d.rank <= 64 && p->tile_rows == 32) ||
        (p->tile_rows != 8 && p->tile_rows != 16 && p->tile_rows != 32))
      p->tile_rows = 0;
  }
  if (const char* form = std::getenv("LGT_GEMM_ADAPTERS_FORM"); form && *form) p->form = std::atoi(form);
  if (cudaGetDevice(&p->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&p->sms, cudaDevAttrMultiProcessorCount, p->device) != cudaSuccess) {
    cudaGetLastError();
    p->device = -1;
  } else if (cudaMalloc(&p->d_status, 16) != cudaSuccess || cudaMemset(p->d_status, 0, 16) != cudaSuccess) {
    cudaGetLastError();
    if (p->d_status) cudaFree(p->d_status);
    delete p;
    return GEMM_ERR_CUDA;
  }
  p->resident[0] = p->sms;
  for (unsigned i = 1; p->device >= 0 && i < 4; ++i) {
    p->resident[i] = d.dtype == GEMM_BF16 ? lgt::resident_adapter_clusters<true>(1u << i) : lgt::resident_adapter_clusters<false>(1u << i);
    if (p->resident[i] < 0) {
      cudaGetLastError();
      cudaFree(p->d_status);
      delete p;
      return GEMM_ERR_CUDA;
    }
  }
  *plan = p;
  return GEMM_OK;
}

gemm_status_t gemm_adapters_run(gemm_adapters_plan_t* plan, const void* x, int64_t x_stride, const void* A, const void* B,
                                const float* scales, const int32_t* offsets, const int32_t* order, int64_t rows,
                                const void* base, int64_t base_stride, void* out, int64_t out_stride, void* stream) {
  using namespace lgt;
  if (!plan || rows < 0) return GEMM_ERR_INVALID_ARG;
  const gemm_adapters_desc_t& d = plan->d;
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
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  if (dev != plan->device) return GEMM_ERR_INVALID_ARG;  // (the status word is there)
  const int sms = plan->sms;
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
  a.ctas = 1;
  const int64_t busy = std::min<int64_t>(d.groups, rows);
  const bool bf16 = d.dtype == GEMM_BF16;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  // The two forms' times, in us, from their rounds of tiles (measured at K = N =
  // 4096).  The sizes of the groups are not known here: as many of them have rows as
  // if every row had chosen one by itself, and half a tile of each is counted as empty
  // (834 rows of 54 groups, rank 88, 2536 x 1832, in the first form 24 us, with four
  // CTAs a tile, which 35 tiles would allow, 50).
  // The form for few rows: a CTA by itself takes so long for a tile with two on an SM
  // (but 1 us), 3/4 of that with one; a cluster its share, and 0.3 us a CTA for the joins.  4 us (8
  // above a rank of 64) come to it.  Small tiles read the group's matrices more often,
  // from L2, but there are more of them (64 rows of 4 groups, rank 64: 8 rows a tile 8.9
  // us, 16 10.7; 4096 rows of 100, rank 24: 47, 33, 32 rows a tile 51).  0: no such
  // kernel, since it was nowhere the fastest.
  static constexpr double kTileUs[4][3] = {{12.5, 21.0, 38.0}, {20.0, 27.0, 52.0}, {29.0, 50.0, 0.0}, {60.0, 0.0, 68.0}};
  const int mt = d.rank <= 16 ? 0 : d.rank <= 32 ? 1 : d.rank <= 64 ? 2 : 3;
  const double with_rows = d.groups * (1.0 - std::exp(-static_cast<double>(rows) / d.groups));
  auto tiles_of = [&](int64_t height) {
    return static_cast<int64_t>(std::max(with_rows, static_cast<double>(rows) / static_cast<double>(height) + with_rows / 2) + 0.5);
  };
  const double row_bytes = 2.0 * static_cast<double>(d.K + 2 * d.N), scale = row_bytes / (2.0 * 3 * 4096);
  int nt = 1;
  double best_us = 1e30;
  for (int i = 2; i >= 0; --i) {
    if (kTileUs[mt][i] == 0.0 || (plan->tile_rows > 0 && plan->tile_rows != 8 << i)) continue;
    const int on_sm = i == 2 && mt == 3 ? 1 : 2;
    for (int lg = 0; lg < 4 && (lg == 0 || std::max(d.N, d.K) >= int64_t{256} << lg); ++lg) {
      // (as many clusters run at once as of the other form, on each CTA that an SM has room for)
      const double clusters = static_cast<double>(tiles_of(8 << i)), rounds = clusters / (on_sm * plan->resident[lg]);
      if (lg > 0 && rounds > 1.0) break;
      double tile_us = std::max(1.0, kTileUs[mt][i] * scale / (1 << lg));
      if (rounds > 1.0)
        tile_us *= (std::ceil(rounds - 0.05) + 1.1 * rounds) / 2;
      else if (on_sm == 2 && clusters * (1 << lg) <= sms)
        tile_us *= 0.75;
      const double us = (mt == 3 ? 8.0 : 4.0) + (lg > 0 ? 0.3 * (1 << lg) : 0.0) + tile_us;
      if (us < best_us) {
        best_us = us;
        nt = 1 << i;
        a.ctas = 1u << lg;
      }
    }
  }
  const int64_t tiles = rows / (8 * nt) + busy + 1;  // (at most, those of rows of no group among them)
  // The form for many rows: an SM moves 60 bytes a ns (45 where it gathers), a tile's
  // ends are as long as 16 rows, all SMs together move 6.1 TB/s, and the exchange of
  // parts takes 3 us and 0.1 us x CTAs^2 for every 16 of the rank.
  const int64_t rank16 = (d.rank + 15) / 16;
  const double all_us = static_cast<double>(rows) * row_bytes / 6.1e6;
  int lg = -1;
  uint32_t height = kAtcRows;
  for (int i = 0; i < 4 && (rows > 8 * busy || plan->form > 0); ++i) {
    const int64_t at_once = plan->resident[i];
    if (at_once < 1 || d.K < static_cast<int64_t>(TILE_K) << i || d.N < int64_t{128} << i) break;
    // Tiles as high as fill the last round best (a round is bound by what one SM moves:
    // 16384 rows of 8 groups, rank 64, in 132 tiles of 128 rows 77 us, in 150 of 112 75.8;
    // 12000 of 6 in 108 of 128 68.8, in 138 of 96 63.8).
    uint32_t h = kAtcRows;
    int64_t rounds = 0, least = 0;
    for (uint32_t x = kAtcRows; x >= 64; x -= 16) {
      const int64_t r = (tiles_of(x) + static_cast<int64_t>(std::sqrt(with_rows / 3)) + at_once - 1) / at_once, cost = r * (x + 16);
      if (x == kAtcRows || cost < least) {
        least = cost;
        rounds = r;
        h = x;
      }
    }
    const double tile_us = (h + 16) * row_bytes / (order ? 45e3 : 60e3) / (1 << i) + (i > 0 ? 0.1 * static_cast<double>(rank16 << (2 * i)) : 0.0);
    const double us = (i > 0 ? 12.0 : 9.0) + std::max(all_us, static_cast<double>(rounds) * tile_us);
    if (plan->form < 0 ? us < best_us : plan->form == 1 << i) {
      best_us = us;
      lg = i;
      height = h;
    }
  }
  cudaError_t e;
  if (lg >= 0) {
    AdapterTcArgs t;
    t.p = a;
    t.status = plan->d_status;
    // (a wait may be for all of a tile's blocks)
    t.wait_limit_ns = plan->wait_limit_ns + static_cast<uint64_t>(d.K / TILE_K + d.N / 128) * 4000;
    t.rank16 = static_cast<uint32_t>(rank16);
    t.chunks = (t.rank16 + 3) / 4;
    t.height = height;
    t.stage_bytes = kAtcTile + t.rank16 * 16 * 128;
    const uint32_t tables = kAtcBars * 8 + 1544 + 256 + 8 * static_cast<uint32_t>(d.groups + 1);
    t.stages = std::min<uint32_t>(kAtcMaxStages, (kAtcSmem - 1024 - kAtcStaging - tables) / t.stage_bytes);
    // (a rank of one stretch leaves room for the parts behind u and B, one of two has them in B's place)
    t.parts = t.chunks == 1 ? 4 * kAtcTile : 2 * t.chunks * kAtcTile;
    t.region = std::max(t.stages * t.stage_bytes, t.chunks == 1 ? t.parts + kAtcRows * t.rank16 * 64 : 4 * t.chunks * kAtcTile);
    t.idesc_u = idesc_f16(bf16, 0u, 0u, kAtcRows, t.rank16 * 16);
    t.idesc_out = idesc_f16(bf16, 0u, 0u, kAtcRows, 0u);
    t.withhold = plan->withhold_armed ? __atomic_exchange_n(&plan->withhold_armed, 0, __ATOMIC_ACQ_REL) : 0;
    if (!encode_x(&t.tm_x, x, bf16, d.K, rows, x_stride, order ? 1 : height) ||
        !encode_dense(&t.tm_a, A, bf16, d.K, d.rank, d.groups, t.rank16 * 16) ||
        !encode_dense(&t.tm_b, B, bf16, d.rank, d.N, d.groups, 128))
      return GEMM_ERR_CUDA;
    t.p.ctas = 1u << lg;
    const unsigned clusters = static_cast<unsigned>(std::min<int64_t>(rows / height + busy + 1, plan->resident[lg]));
    e = bf16 ? launch_adapters_tc<true>(t, clusters, s) : launch_adapters_tc<false>(t, clusters, s);
  } else {
    const unsigned clusters = static_cast<unsigned>(std::min<int64_t>(tiles, 2 * sms / a.ctas));
    e = bf16 ? launch_adapters<true>(a, nt, clusters, s) : launch_adapters<false>(a, nt, clusters, s);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  return GEMM_OK;
}

gemm_status_t gemm_adapters_sync_status(gemm_adapters_plan_t* plan, void* stream) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  if (!plan->d_status) return GEMM_ERR_CUDA;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return GEMM_ERR_CUDA;
  lgt::DeviceStatus st;
  if (cudaMemcpy(&st, plan->d_status, sizeof(st), cudaMemcpyDeviceToHost) != cudaSuccess) return GEMM_ERR_CUDA;
  if (st.code != 0) {
    if (cudaMemset(plan->d_status, 0, sizeof(st)) != cudaSuccess) return GEMM_ERR_CUDA;
    return static_cast<gemm_status_t>(st.code);
  }
  return GEMM_OK;
}

gemm_status_t gemm_adapters_withhold_load(gemm_adapters_plan_t* plan) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  __atomic_store_n(&plan->withhold_armed, 1, __ATOMIC_RELEASE);
  return GEMM_OK;
}

gemm_status_t gemm_adapters_destroy(gemm_adapters_plan_t* plan) {
  if (!plan) return GEMM_OK;
  if (plan->d_status) cudaFree(plan->d_status);
  delete plan;
  return GEMM_OK;
}

}  // extern "C"
