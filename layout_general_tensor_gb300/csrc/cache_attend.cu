// Attention of one query a sequence over the paged 8-bit cache
// (include/attn_cache.h).
//
// Bound: memory, the codes of every key and value read once; the arithmetic
// per byte is small (2 * group multiply-adds), so warp-level matrix
// instructions on registers carry it and nothing goes through shared memory
// on the way.
//
// Work.  A tile is 64 keys of one sequence and key head.  The tiles of the
// whole batch, in the order (sequence, head, key), are cut into as many equal
// runs as there are CTAs, so a long sequence among short ones spreads over
// the GPU and every CTA reads the same number of bytes.  Each CTA finds its
// run from the lengths by a prefix sum in shared memory.  Only the first and
// the last sequence-head of a run can be shared with other CTAs; their
// unnormalised results go to the workspace, and the CTA that arrives last
// on the sequence-head's counter joins them, in the order of the keys.
//
// A warp takes 16 keys at a time (always inside one page).  With G <= 8 query
// heads to a key head (NT = 1; 16 with NT = 2):
//   S^T = K Q^T    m16n8k16, 16 keys x 8 heads; the contraction over d may
//                  take d in any order common to both, so a lane's fragments
//                  are four consecutive codes of a 16-byte load.
//   O^T += V^T P^T m16n8k16, 16 values of d x 8 heads over 16 keys; a lane
//                  loads the same bytes of four keys, and one byte permute
//                  pairs two keys' codes before they are widened, so V is
//                  transposed on the way for nothing.
// e4m3 codes widen to fp16 exactly.  The keys' powers of two multiply the
// logits; the values' multiply the weights: with t the logit in log2 units
// and e the value's power, the sum l takes p = 2^(t - m) and the product
// w = 2^(t - m + e - R), an integer R of its own so that w is p times a power
// of two; m and R are moved only when something exceeds them by 2^8.  So w
// spans fp16 whatever the rows' magnitudes are, and the largest contribution
// to the result is the one that is held most exactly.  The result is the
// product's sum times 2^R / l.
#include <cmath>
#include <cstdint>

#include "cache.h"
#include "half_types.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace lgt {
namespace {

constexpr int kAtWarps = 8;
constexpr int kAtThreads = kAtWarps * 32;
constexpr int kAtTile = 64;         // keys
constexpr int kAtMaxBatch = 8192;   // prefix sums in shared memory
constexpr float kAtLazy = 8.0f;

struct AttendArgs {
  const uint8_t *k, *v, *ke, *ve;
  const uint16_t* q;
  uint16_t* out;
  const int32_t *table, *lengths;
  float* part;        // [cta][2][heads][D + 4]: sums, then l, m, R
  int32_t* counters;  // one per (sequence, key head, head group)
  int64_t qs, os, table_stride;
  uint32_t pages;
  int32_t max_pages, batch, hk, group, hgroups;  // hgroups: groups of 8 * NT query heads of a key head
  int32_t max_len;
  MagicDiv div_page;
  float cs;  // scale * log2(e)
  int32_t page;
};

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Two e4m3 codes (the low or the high half of a word) as two fp16 values.
__device__ __forceinline__ uint32_t widen_lo(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t widen_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

// 2^e for an integer e in [-126, 127], clamped below to 0.
__device__ __forceinline__ float pow2i(int e) {
  return e < -126 ? 0.0f : __uint_as_float(static_cast<uint32_t>(min(e, 127) + 127) << 23);
}

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Joining partial results {l, m, R}: R against the common m, and the factors
// of l and of the sum.  A part that saw no keys (m never set) counts nothing.
template <typename P>
__device__ __forceinline__ float ref_at(P s, float m) {
  return s[1] == -INFINITY ? -INFINITY : s[1] - m + s[2];
}
template <typename P>
__device__ __forceinline__ float l_scale(P s, float m) {
  return s[1] == -INFINITY ? 0.0f : ex2f(s[1] - m);
}
template <typename P>
__device__ __forceinline__ float sum_scale(P s, float m, float R) {
  return s[1] == -INFINITY ? 0.0f : ex2f(s[1] - m + s[2] - R);
}

template <int D, int NT, bool BF16>
__global__ void __launch_bounds__(kAtThreads, NT == 1 ? 2 : 1) cache_attend_kernel(const __grid_constant__ AttendArgs a) {
  constexpr int HP = 8 * NT;       // query heads of a pass
  constexpr int ROW = D + 4;       // floats of a partial row
  constexpr int KP = D / 64;       // 16-byte pieces of a key a lane loads
  constexpr int VW = D / 32;       // words of a value row a lane loads (D / 8 bytes)
  constexpr int MT = D / 16;       // m-tiles of O^T
  extern __shared__ uint32_t smem_u[];
  float* red = reinterpret_cast<float*>(smem_u);             // [warp][HP][ROW]
  uint32_t* prefix = smem_u + kAtWarps * HP * ROW;           // batch + 1
  __shared__ uint32_t scan[kAtWarps];
  __shared__ int last_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  pdl_launch_dependents();
  pdl_wait();

  // ---- prefix sums of the sequences' tiles (at least one each: somebody writes the zeros)
  const uint32_t per_seq = static_cast<uint32_t>(a.hk * a.hgroups);
  {
    uint32_t carry = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kAtThreads) {
      const int b = b0 + static_cast<int>(threadIdx.x);
      uint32_t n = 0;
      if (b < a.batch) {
        const int len = min(max(a.lengths[b], 0), a.max_len);
        n = static_cast<uint32_t>(max((len + kAtTile - 1) / kAtTile, 1)) * per_seq;
      }
      uint32_t x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) scan[warp] = x;
      __syncthreads();
      uint32_t before = carry, all = 0;
#pragma unroll
      for (int w = 0; w < kAtWarps; ++w) {
        before += w < warp ? scan[w] : 0u;
        all += scan[w];
      }
      if (b < a.batch) prefix[b] = before + x - n;
      carry += all;
      __syncthreads();
    }
    if (threadIdx.x == 0) prefix[a.batch] = carry;
    __syncthreads();
  }
  // (never more CTAs than tiles: every run has a tile, so every CTA between a
  // sequence-head's first and last takes part in it)
  const uint32_t total = prefix[a.batch], ctas = min(gridDim.x, total);
  if (blockIdx.x >= ctas) return;
  auto run_start = [&](uint32_t cta) { return static_cast<uint32_t>(static_cast<uint64_t>(cta) * total / ctas); };
  auto owner = [&](uint32_t tile) {
    return static_cast<uint32_t>((static_cast<uint64_t>(tile + 1) * ctas - 1) / total);
  };
  const uint32_t t0 = run_start(blockIdx.x), t1 = run_start(blockIdx.x + 1);
  int b = 0;
  {
    int lo = 0, hi = a.batch - 1;  // the last sequence whose prefix is <= t0
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= t0) lo = mid; else hi = mid - 1;
    }
    b = lo;
  }

  for (uint32_t t = t0; t < t1;) {
    while (t >= prefix[b + 1]) ++b;
    const int len = min(max(a.lengths[b], 0), a.max_len);
    const uint32_t tiles = (prefix[b + 1] - prefix[b]) / per_seq;  // of one pass over the keys
    const uint32_t in_seq = t - prefix[b];
    const uint32_t hh = in_seq / tiles, tile = in_seq - hh * tiles;
    const int h = static_cast<int>(hh) / a.hgroups, hg = static_cast<int>(hh) - h * a.hgroups;
    const uint32_t seg_end = min(t1, prefix[b] + (hh + 1) * tiles);
    const int key0 = static_cast<int>(tile) * kAtTile;
    const int key1 = min(len, static_cast<int>(tile + (seg_end - t)) * kAtTile);
    const int heads = min(HP, a.group - hg * HP);  // of this pass
    const int hq0 = h * a.group + hg * HP;

    // ---- the queries as B fragments: lane (r, c) has head r's values
    // p*64 + c*16 + 4j + {0, 1 | 2, 3} for step (p, j), in fp16 (bf16 ones
    // times a power of two that brings the head's largest to [1, 2))
    uint32_t qf[NT][KP * 4][2];
    float qscale[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int head = n * 8 + r;
      uint4 w[KP][2];
#pragma unroll
      for (int p = 0; p < KP; ++p)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          w[p][e] = make_uint4(0u, 0u, 0u, 0u);
          if (head < heads)
            w[p][e] = *reinterpret_cast<const uint4*>(a.q + static_cast<int64_t>(b) * a.qs +
                                                      static_cast<int64_t>(hq0 + head) * D + p * 64 + c * 16 + e * 8);
        }
      float mine = a.cs;
      float inv = 1.0f;
      if constexpr (BF16) {
        uint32_t top = 0;  // the largest exponent field of a finite value
#pragma unroll
        for (int p = 0; p < KP; ++p)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t x[4] = {w[p][e].x, w[p][e].y, w[p][e].z, w[p][e].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t e0 = (x[i] >> 7) & 0xffu, e1 = (x[i] >> 23) & 0xffu;
              top = max(top, max(e0 == 255u ? 0u : e0, e1 == 255u ? 0u : e1));
            }
          }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = max(static_cast<int>(top), 1) - 127;
        inv = pow2i(-max(e, -126));
        mine = a.cs * pow2i(e);
      }
#pragma unroll
      for (int p = 0; p < KP; ++p)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 src = w[p][j >> 1];
          const uint32_t w0 = (j & 1) ? src.z : src.x, w1 = (j & 1) ? src.w : src.y;
          if constexpr (BF16) {
            const float2 x0 = unpack_pair16<true>(w0), x1 = unpack_pair16<true>(w1);
            qf[n][p * 4 + j][0] = pack_pair16<false>(x0.x * inv, x0.y * inv);
            qf[n][p * 4 + j][1] = pack_pair16<false>(x1.x * inv, x1.y * inv);
          } else {
            qf[n][p * 4 + j][0] = w0;
            qf[n][p * 4 + j][1] = w1;
          }
        }
      // this lane's columns of S are heads 2c and 2c + 1
      qscale[n][0] = __shfl_sync(0xffffffffu, mine, 8 * c);
      qscale[n][1] = __shfl_sync(0xffffffffu, mine, 8 * c + 4);
    }

    float o[MT][NT][4];
    float l[NT][2], m[NT][2], R[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      l[n][0] = l[n][1] = 0.0f;
      m[n][0] = m[n][1] = R[n][0] = R[n][1] = -INFINITY;
#pragma unroll
      for (int i = 0; i < MT; ++i) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.0f;
    }

    // ---- the keys, 16 at a time
    uint4 kw[2][KP];
    uint32_t vw[4][VW];
    int kx[2], vx[2];
    auto page_of = [&](int key) -> uint32_t {
      if (key >= key1) return 0xffffffffu;
      return static_cast<uint32_t>(
          a.table[static_cast<int64_t>(b) * a.table_stride + magic_div(static_cast<uint32_t>(key), a.div_page)]);
    };
    auto row_of = [&](int key, uint32_t page) -> int64_t {
      const int off = key - static_cast<int>(magic_div(static_cast<uint32_t>(key), a.div_page)) * a.page;
      return (static_cast<int64_t>(page) * a.hk + h) * a.page + off;
    };
    auto load_k = [&](int key, uint32_t page) {
      if (page >= a.pages) return;
      const int64_t row = row_of(key, page);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int p = 0; p < KP; ++p) kw[i][p] = ld_stream_v4(a.k + (row + r + 8 * i) * D + p * 64 + c * 16);
        kx[i] = a.ke[row + r + 8 * i];
      }
    };
    auto load_v = [&](int key, uint32_t page) {
      if (page >= a.pages) return;
      const int64_t row = row_of(key, page);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* p = a.v + (row + 2 * c + (i & 1) + 8 * (i >> 1)) * D + r * (D / 8);
        if constexpr (D == 128) {
          const uint4 x = ld_stream_v4(p);
          vw[i][0] = x.x; vw[i][1] = x.y; vw[i][2] = x.z; vw[i][3] = x.w;
        } else {
          const uint2 x = ld_stream_v2(p);
          vw[i][0] = x.x; vw[i][1] = x.y;
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) vx[i] = a.ve[row + r + 8 * i];
    };

    int key = key0 + warp * 16;
    uint32_t page = page_of(key), next_page = page_of(key + kAtWarps * 16);
    if (key < key1) {
      load_k(key, page);
      load_v(key, page);
    }
    for (; key < key1; key += kAtWarps * 16) {
      const int next = key + kAtWarps * 16;
      const uint32_t page2 = page_of(next + kAtWarps * 16);
      const int valid = page < a.pages ? min(16, key1 - key) : 0;  // a page that is none holds no keys
      if (valid > 0) {
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
        for (int p = 0; p < KP; ++p) {
          const uint32_t x0[4] = {kw[0][p].x, kw[0][p].y, kw[0][p].z, kw[0][p].w};
          const uint32_t x1[4] = {kw[1][p].x, kw[1][p].y, kw[1][p].z, kw[1][p].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t a0 = widen_lo(x0[j]), a1 = widen_lo(x1[j]), a2 = widen_hi(x0[j]), a3 = widen_hi(x1[j]);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_16816(s[n], a0, a1, a2, a3, qf[n][p * 4 + j][0], qf[n][p * 4 + j][1]);
          }
        }
        const int k0e = kx[0], k1e = kx[1];
        const float v0e = static_cast<float>(vx[0] - 127), v1e = static_cast<float>(vx[1] - 127);
        load_k(next, next_page);
        const float f0 = pow2i(k0e - 127), f1 = pow2i(k1e - 127);
        bool over = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          s[n][0] = r < valid ? s[n][0] * f0 * qscale[n][0] : -INFINITY;
          s[n][1] = r < valid ? s[n][1] * f0 * qscale[n][1] : -INFINITY;
          s[n][2] = r + 8 < valid ? s[n][2] * f1 * qscale[n][0] : -INFINITY;
          s[n][3] = r + 8 < valid ? s[n][3] * f1 * qscale[n][1] : -INFINITY;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float ref = m[n][e] == -INFINITY ? 0.0f : m[n][e];
            const float d0 = s[n][e] - ref, d1 = s[n][2 + e] - ref, top = R[n][e] + kAtLazy;
            over |= d0 > kAtLazy || d1 > kAtLazy || d0 + v0e > top || d1 + v1e > top;
          }
        }
        if (__any_sync(0xffffffffu, over)) {
          // move the references to these keys' maxima, where they are larger
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float x = fmaxf(s[n][e], s[n][2 + e]);
#pragma unroll
              for (int sh = 4; sh < 32; sh <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, sh));
              const float mn = fmaxf(m[n][e], x), ref = mn == -INFINITY ? 0.0f : mn;
              float y = fmaxf(s[n][e] - ref + v0e, s[n][2 + e] - ref + v1e);
#pragma unroll
              for (int sh = 4; sh < 32; sh <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, sh));
              const float moved = m[n][e] == -INFINITY ? -INFINITY : m[n][e] - ref;  // <= 0
              const float old = m[n][e] == -INFINITY ? -INFINITY : R[n][e] + moved;  // R against the new m
              const float Rn = fmaxf(rintf(old), ceilf(y));
              const float fl = ex2f(moved), fo = m[n][e] == -INFINITY ? 0.0f : ex2f(old - Rn);
              l[n][e] *= fl;
              m[n][e] = mn;
              R[n][e] = Rn;
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                o[i][n][e] *= fo;
                o[i][n][2 + e] *= fo;
              }
            }
        }
        uint32_t pf[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float ref = m[n][e] == -INFINITY ? 0.0f : m[n][e];
            const float p0 = ex2f(s[n][e] - ref), p1 = ex2f(s[n][2 + e] - ref);
            l[n][e] += p0 + p1;
            // (R never set: every p is 0 or not a number)
            const float down = m[n][e] == -INFINITY ? 0.0f : R[n][e];
            w[e] = p0 * pow2i(static_cast<int>(v0e - down));
            w[2 + e] = p1 * pow2i(static_cast<int>(v1e - down));
          }
          pf[n][0] = transpose_8x8(pack_pair16<false>(w[0], w[1]));
          pf[n][1] = transpose_8x8(pack_pair16<false>(w[2], w[3]));
        }
        if (valid < 16) {  // what lies past the end may be anything, a NaN too
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (2 * c + (i & 1) + 8 * (i >> 1) >= valid) {
#pragma unroll
              for (int j = 0; j < VW; ++j) vw[i][j] = 0u;
            }
        }
#pragma unroll
        for (int j = 0; j < VW; ++j) {
          const uint32_t lo0 = prmt(vw[0][j], vw[1][j], 0x5140u), lo1 = prmt(vw[0][j], vw[1][j], 0x7362u);
          const uint32_t hi0 = prmt(vw[2][j], vw[3][j], 0x5140u), hi1 = prmt(vw[2][j], vw[3][j], 0x7362u);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t x = e ? lo1 : lo0, y = e ? hi1 : hi0;
            const uint32_t a0 = widen_lo(x), a1 = widen_hi(x), a2 = widen_lo(y), a3 = widen_hi(y);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_16816(o[2 * j + e][n], a0, a1, a2, a3, pf[n][0], pf[n][1]);
          }
        }
      } else {
        load_k(next, next_page);
      }
      load_v(next, next_page);
      page = next_page;
      next_page = page2;
    }

    // ---- the warps' results together, in the order of the warps
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], sh);
        float* row = red + (warp * HP + n * 8 + 2 * c + e) * ROW;
        if (r == 0) {
          row[D] = l[n][e];
          row[D + 1] = m[n][e];
          row[D + 2] = R[n][e];
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          row[r * (D / 8) + 2 * i] = o[i][n][e];
          row[r * (D / 8) + 2 * i + 1] = o[i][n][2 + e];
        }
      }
    __syncthreads();
    const uint32_t first_tile = prefix[b] + hh * tiles, last_tile = first_tile + tiles - 1;
    const uint32_t c0 = owner(first_tile), c1 = owner(last_tile);
    auto write_out = [&](int head, int d, float acc, float lt, float Rt) {
      const float y = lt == 0.0f ? 0.0f : acc * (ex2f(Rt) / lt);
      uint16_t* dst = a.out + static_cast<int64_t>(b) * a.os + static_cast<int64_t>(hq0 + head) * D + d;
      *dst = static_cast<uint16_t>(pack_pair16<BF16>(y, 0.0f));
    };
    for (int i = threadIdx.x; i < heads * D; i += kAtThreads) {
      const int head = i / D, d = i - head * D;
      const float* rows = red + head * ROW;
      float mt = -INFINITY, Rt = -INFINITY;
#pragma unroll
      for (int w = 0; w < kAtWarps; ++w) mt = fmaxf(mt, rows[w * HP * ROW + D + 1]);
#pragma unroll
      for (int w = 0; w < kAtWarps; ++w) Rt = fmaxf(Rt, ref_at(rows + w * HP * ROW + D, mt));
      float acc = 0.0f, lt = 0.0f;
#pragma unroll
      for (int w = 0; w < kAtWarps; ++w) {
        const float* row = rows + w * HP * ROW;
        acc += row[d] * sum_scale(row + D, mt, Rt);
        lt += row[D] * l_scale(row + D, mt);
      }
      if (c0 == c1) {
        write_out(head, d, acc, lt, Rt);
      } else {
        float* row = a.part + ((static_cast<int64_t>(blockIdx.x) * 2 + (t == t0 ? 0 : 1)) * HP + head) * ROW;
        row[d] = acc;
        if (d == 0) {
          row[D] = lt;
          row[D + 1] = mt;
          row[D + 2] = Rt;
        }
      }
    }
    if (c0 != c1) {
      __threadfence();
      __syncthreads();
      int32_t* counter = a.counters + static_cast<int64_t>(b) * per_seq + hh;
      if (threadIdx.x == 0) last_flag = atomicAdd(counter, 1) == static_cast<int>(c1 - c0);
      __syncthreads();
      if (last_flag) {
        __threadfence();
        if (threadIdx.x == 0) *counter = 0;
        for (int i = threadIdx.x; i < heads * D; i += kAtThreads) {
          const int head = i / D, d = i - head * D;
          auto row_at = [&](uint32_t cta) -> const volatile float* {  // (other CTAs wrote it: not through L1)
            const int slot = cta == c0 && run_start(c0) != first_tile ? 1 : 0;
            return a.part + ((static_cast<int64_t>(cta) * 2 + slot) * HP + head) * ROW;
          };
          float mt = -INFINITY, Rt = -INFINITY;
          for (uint32_t x = c0; x <= c1; ++x) mt = fmaxf(mt, row_at(x)[D + 1]);
          for (uint32_t x = c0; x <= c1; ++x) Rt = fmaxf(Rt, ref_at(row_at(x) + D, mt));
          float acc = 0.0f, lt = 0.0f;
          for (uint32_t x = c0; x <= c1; ++x) {
            const volatile float* row = row_at(x);
            acc += row[d] * sum_scale(row + D, mt, Rt);
            lt += row[D] * l_scale(row + D, mt);
          }
          write_out(head, d, acc, lt, Rt);
        }
      }
    }
    __syncthreads();  // red and last_flag are used again by the next segment
    t = seg_end;
  }
}

struct AttendPlan {
  int nt, hgroups, ctas;
  size_t part_bytes, bytes;
};

// CTAs: two an SM where the registers allow it (up to eight heads a pass).
bool plan_attend(int32_t q_heads, int32_t k_heads, int32_t head_dim, int32_t batch, AttendPlan* p) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  const int group = q_heads / k_heads;
  p->nt = group <= 8 ? 1 : 2;
  p->hgroups = (group + 8 * p->nt - 1) / (8 * p->nt);
  p->ctas = sms * (p->nt == 1 ? 2 : 1);
  p->part_bytes = static_cast<size_t>(p->ctas) * 2 * 8 * p->nt * (head_dim + 4) * sizeof(float);
  p->bytes = p->part_bytes + static_cast<size_t>(batch) * k_heads * p->hgroups * sizeof(int32_t);
  return true;
}

template <int D, int NT, bool BF16>
cudaError_t launch_attend(const AttendArgs& a, int ctas, cudaStream_t stream) {
  const size_t smem = sizeof(uint32_t) * (static_cast<size_t>(kAtWarps) * 8 * NT * (D + 4) + a.batch + 1);
  constexpr size_t most = sizeof(uint32_t) * (static_cast<size_t>(kAtWarps) * 8 * NT * (D + 4) + kAtMaxBatch + 1);
  const cudaError_t e = set_smem_once<cache_attend_kernel<D, NT, BF16>>(static_cast<int>(most));
  if (e != cudaSuccess) return e;
  return launch_pdl(cache_attend_kernel<D, NT, BF16>, dim3(static_cast<unsigned>(ctas)), dim3(kAtThreads), smem, stream, a);
}

bool attend_shape_ok(int32_t q_heads, int32_t k_heads, int32_t head_dim, int32_t batch) {
  return q_heads >= 1 && k_heads >= 1 && q_heads % k_heads == 0 && (head_dim == 64 || head_dim == 128) && batch >= 0;
}

}  // namespace
}  // namespace lgt

extern "C" gemm_status_t attn_cache_attend_workspace_size(int32_t q_heads, int32_t k_heads, int32_t head_dim,
                                                          int32_t batch, size_t* bytes) {
  if (!bytes || !lgt::attend_shape_ok(q_heads, k_heads, head_dim, batch)) return GEMM_ERR_INVALID_ARG;
  *bytes = 0;
  if (batch > lgt::kAtMaxBatch) return GEMM_ERR_UNSUPPORTED;
  lgt::AttendPlan p;
  if (!lgt::plan_attend(q_heads, k_heads, head_dim, batch, &p)) return GEMM_ERR_CUDA;
  *bytes = p.bytes;
  return GEMM_OK;
}

extern "C" gemm_status_t attn_cache_attend(const attn_cache_t* cache, const void* Q, int64_t q_stride, int32_t q_heads,
                                           const int32_t* page_table, int64_t table_stride, int32_t max_pages,
                                           const int32_t* lengths, int32_t batch, float scale, int32_t dtype, void* out,
                                           int64_t out_stride, void* workspace, size_t workspace_bytes, void* stream) {
  if (!cache || !lgt::cache_ok(*cache) || (dtype != GEMM_F16 && dtype != GEMM_BF16)) return GEMM_ERR_INVALID_ARG;
  const attn_cache_t& c = *cache;
  if (!lgt::attend_shape_ok(q_heads, c.k_heads, c.head_dim, batch)) return GEMM_ERR_INVALID_ARG;
  if (!(scale >= 0.0f) || std::isinf(scale)) return GEMM_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(q_heads) * c.head_dim;
  if (q_stride == 0) q_stride = row;
  if (out_stride == 0) out_stride = row;
  if (table_stride == 0) table_stride = max_pages;
  if (q_stride < row || out_stride < row || q_stride % 8 != 0 || out_stride % 8 != 0 || max_pages < 0 ||
      table_stride < max_pages)
    return GEMM_ERR_INVALID_ARG;
  if (batch == 0) return GEMM_OK;
  if (!Q || !out || !lengths || (!page_table && max_pages > 0)) return GEMM_ERR_INVALID_ARG;
  for (const void* p : {Q, static_cast<const void*>(out), static_cast<const void*>(c.k), static_cast<const void*>(c.v)})
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return GEMM_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(lengths) | reinterpret_cast<uintptr_t>(page_table)) % 4 != 0) return GEMM_ERR_ALIGNMENT;
  // (tiles are counted in 32 bits, keys in 31)
  const int64_t max_len = static_cast<int64_t>(max_pages) * c.page_size;
  if (batch > lgt::kAtMaxBatch || max_len > (int64_t{1} << 30)) return GEMM_ERR_UNSUPPORTED;
  lgt::AttendPlan p;
  if (!lgt::plan_attend(q_heads, c.k_heads, c.head_dim, batch, &p)) return GEMM_ERR_CUDA;
  if ((max_len / lgt::kAtTile + 1) * batch * c.k_heads * p.hgroups >= (int64_t{1} << 31)) return GEMM_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < p.bytes || reinterpret_cast<uintptr_t>(workspace) % 16 != 0)
    return GEMM_ERR_WORKSPACE;
  lgt::AttendArgs a;
  a.k = static_cast<const uint8_t*>(c.k);
  a.v = static_cast<const uint8_t*>(c.v);
  a.ke = static_cast<const uint8_t*>(c.k_exp);
  a.ve = static_cast<const uint8_t*>(c.v_exp);
  a.q = static_cast<const uint16_t*>(Q);
  a.out = static_cast<uint16_t*>(out);
  a.table = page_table;
  a.lengths = lengths;
  a.part = static_cast<float*>(workspace);
  a.counters = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + p.part_bytes);
  a.qs = q_stride;
  a.os = out_stride;
  a.table_stride = table_stride;
  a.pages = static_cast<uint32_t>(c.pages);
  a.max_pages = max_pages;
  a.batch = batch;
  a.hk = c.k_heads;
  a.group = q_heads / c.k_heads;
  a.hgroups = p.hgroups;
  a.max_len = static_cast<int32_t>(max_len);
  a.div_page = lgt::magic_encode(static_cast<uint32_t>(c.page_size));
  a.cs = (scale > 0.0f ? scale : 1.0f / std::sqrt(static_cast<float>(c.head_dim))) * 1.4426950408889634f;
  a.page = c.page_size;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = dtype == GEMM_BF16;
  cudaError_t e;
  if (c.head_dim == 128)
    e = p.nt == 1 ? (bf16 ? lgt::launch_attend<128, 1, true>(a, p.ctas, s) : lgt::launch_attend<128, 1, false>(a, p.ctas, s))
                  : (bf16 ? lgt::launch_attend<128, 2, true>(a, p.ctas, s) : lgt::launch_attend<128, 2, false>(a, p.ctas, s));
  else
    e = p.nt == 1 ? (bf16 ? lgt::launch_attend<64, 1, true>(a, p.ctas, s) : lgt::launch_attend<64, 1, false>(a, p.ctas, s))
                  : (bf16 ? lgt::launch_attend<64, 2, true>(a, p.ctas, s) : lgt::launch_attend<64, 2, false>(a, p.ctas, s));
  if (e != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  return GEMM_OK;
}
