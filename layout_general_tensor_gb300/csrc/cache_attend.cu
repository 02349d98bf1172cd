// Attention of one query a sequence over the paged 8-bit cache
// (include/attn_cache.h).
//
// Bound: memory, the codes of every key and value read once; the arithmetic
// per byte is small (2 * group multiply-adds), so warp-level matrix
// instructions on registers carry it and nothing goes through shared memory
// on the way.  Measured (32 / 8 heads of 128): 1 sequence of 65536 tokens 30.4
// us, of which the stream takes 20 at 6.7 TB/s, 64 of 1 to 8192 38.1 us (25 at
// a copy's rate), 64 of 2048 53.6 us (74 %); 5 of 1 to 200 (12 / 2 heads of 64)
// 5.9 us, five dependent trips to memory.
//
// Work.  A pass is one sequence, key head and group of up to 8 query heads; its
// units are its blocks of 16 keys and two more for what a pass costs whatever
// its length (64 ragged sequences: 44 us with one, 39.4 with two to four).  The
// units of the whole batch, pass after pass, are cut into as many equal runs as
// there are CTAs, and a CTA's run into one for each warp, so a long sequence
// among short ones spreads over the GPU and
// every warp reads about the same number of bytes, without meeting another
// before the end of its run.  A pass that lies in one warp's run goes straight
// to the output.  Of the others each warp leaves its unnormalised share (at
// most two: its first and its last) in shared memory, where the CTA joins
// them; the shares of passes that cross CTAs go on to the workspace, and the
// CTA that arrives last on the pass's counter joins those.  All are joined in
// the order of the keys.
//
// A warp takes blocks of 16 keys (always inside one page), one at a time at
// head_dim 128 and two at 64, which is 4 KiB on its way either way, and up to
// eight query heads of a key head; more heads are further passes over the
// keys, which find them in L2 (16 heads in one pass need twice the registers,
// so half the warps: 33 us against 26.5 at 4 x 16384 tokens, 48 / 3 heads).
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
// m is a logit, not rounded to a whole number: so the largest weight of a short
// or peaked row is 1 exactly.  (Rounded up, a sequence alone and in a batch
// differed in 0.3 % of its values instead of up to a third, but the error of a
// sequence of 9 keys beside one of 8962 was 1.9e-4 instead of 4e-6.)
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "cache.h"
#include "half_types.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace lgt {
namespace {

constexpr int kAtWarps = 16;        // of 128 registers: they fill an SM
constexpr int kAtThreads = kAtWarps * 32;
constexpr int kAtHeads = 8;         // query heads of a pass
constexpr int kAtKeys = 16;         // a unit
constexpr int kAtMaxDim = 128;
constexpr int kAtPassUnits = 2;     // of a pass besides its keys
constexpr uint32_t kAtWhole = 4;    // units a warp above an even share up to which passes are not cut among CTAs
constexpr int kAtMaxBatch = 8192;   // lengths and prefix sums in shared memory
constexpr uint32_t kAtJoin = 32;    // CTAs' parts joined in one step; their number is at most its square
constexpr uint32_t kAtNone = 0xffffffffu;
constexpr float kAtLazy = 8.0f;

struct AttendArgs {
  const uint8_t *k, *v, *ke, *ve;
  const uint16_t* q;
  uint16_t* out;
  const int32_t *table, *lengths;
  float* part;        // [cta][2][heads][D + 4]: sums, then l, m, R
  int32_t* counters;  // one per pass, then one per part
  int64_t qs, os, table_stride;
  uint32_t pages;
  int32_t max_pages, batch, hk, group, hgroups;  // hgroups: groups of 8 query heads of a key head
  int32_t max_len;
  MagicDiv div_page, div_seq;  // by the passes of a sequence
  uint32_t each, extra;        // passes of a CTA, and how many have one more, where they are not cut
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

// 2^(exponent byte - 127); of the bytes that no key is written with, 0 gives 0
// and 255 gives 2^127.
__device__ __forceinline__ float key_power(int byte) { return __uint_as_float(static_cast<uint32_t>(min(byte, 254)) << 23); }

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Joining results {l, m, R}, one a lane, over the lanes [first, end] that this
// lane is of: the joint {l, m, R}, and the factor of this lane's sum.  One that
// saw no keys (m never set) counts nothing.
__device__ __forceinline__ float4 join_lanes(float l, float m, float R, int first, int end) {
  const int lane = threadIdx.x & 31;
  auto over = [&](float v, auto op) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float y = __shfl_down_sync(0xffffffffu, v, o);
      if (lane + o <= end) v = op(v, y);
    }
    return __shfl_sync(0xffffffffu, v, first);
  };
  auto most = [](float x, float y) { return fmaxf(x, y); };
  const bool none = m == -INFINITY;
  const float mt = over(m, most);
  const float Rt = over(none ? -INFINITY : m - mt + R, most);
  const float lt = over(l * (none ? 0.0f : ex2f(m - mt)), [](float x, float y) { return x + y; });
  return make_float4(lt, mt, Rt, none ? 0.0f : ex2f(m - mt + R - Rt));
}

// Count this CTA in at `counter`, whose `n`-th arrival sets it back to 0; true
// for that one.  One thread does it after a barrier of the CTA: what the CTA
// wrote before is visible to whoever arrives later, and what the earlier ones
// wrote to it after the next barrier (read past L1).
__device__ __forceinline__ bool arrive_last(int32_t* counter, uint32_t n) {
  int32_t old;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
  if (old != static_cast<int32_t>(n) - 1) return false;
  *counter = 0;
  return true;
}

// Join n <= 32 parts (rows of `heads` heads at their slots) by the whole CTA:
// each thread four values of d of every segs-th part, eight on their way at
// once, while the parts' {l, m, R} are joined, a part a lane.
template <int D, typename SlotOf, typename Put>
__device__ __forceinline__ void join_parts(const float* part, float* smem, uint32_t n, SlotOf slot_of, int heads, Put put) {
  constexpr int ROW = D + 4, HP = kAtHeads, MOST = 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int items = heads * (D / 4);  // at most half of the threads
  const int segs = kAtThreads / items;
  float* factor = smem;                                            // [head][32]
  float4* stats = reinterpret_cast<float4*>(smem + heads * 32);    // [head]
  float4* sums = stats + heads;                                    // [seg][items]
  const int seg = static_cast<int>(threadIdx.x) / items, it = static_cast<int>(threadIdx.x) - seg * items;
  const int head = it / (D / 4), d = it % (D / 4) * 4;
  const bool mine = seg < segs;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
  for (uint32_t p0 = 0; p0 < n; p0 += MOST * segs) {
    float4 x[MOST];
#pragma unroll
    for (int e = 0; e < MOST; ++e) {
      x[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (const uint32_t p = p0 + e * segs + seg; mine && p < n)
        x[e] = __ldcg(reinterpret_cast<const float4*>(part + (slot_of(p) * HP + head) * ROW + d));
    }
    if (p0 == 0) {
      if (warp < heads) {
        float4 st = make_float4(0.0f, -INFINITY, -INFINITY, 0.0f);
        if (lane < static_cast<int>(n))
          st = __ldcg(reinterpret_cast<const float4*>(part + (slot_of(lane) * HP + warp) * ROW + D));
        st = join_lanes(st.x, st.y, st.z, 0, 31);
        factor[warp * 32 + lane] = st.w;
        if (lane == 0) stats[warp] = st;
      }
      __syncthreads();
    }
#pragma unroll
    for (int e = 0; e < MOST; ++e)
      if (const uint32_t p = p0 + e * segs + seg; mine && p < n) {
        const float f = factor[head * 32 + p];
        acc.x += x[e].x * f;
        acc.y += x[e].y * f;
        acc.z += x[e].z * f;
        acc.w += x[e].w * f;
      }
  }
  if (mine) sums[threadIdx.x] = acc;
  __syncthreads();
  if (seg == 0) {
    for (int q = 1; q < segs; ++q) {
      const float4 y = sums[q * items + it];
      acc.x += y.x;
      acc.y += y.y;
      acc.z += y.z;
      acc.w += y.w;
    }
    put(head, d, acc, stats[head]);
  }
  __syncthreads();  // the shared memory is used again
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kAtThreads, 1) cache_attend_kernel(const __grid_constant__ AttendArgs a) {
  constexpr int W = kAtWarps, THREADS = kAtThreads, HP = kAtHeads;
  constexpr int ROW = D + 4;       // floats of a part's row
  constexpr int U = 128 / D;       // blocks of keys a step
  constexpr int KP = D / 64;       // 16-byte pieces of a key a lane loads
  constexpr int VW = D / 32;       // words of a value row a lane loads (D / 8 bytes)
  constexpr int MT = D / 16;       // m-tiles of O^T
  extern __shared__ __align__(16) uint32_t smem_u[];
  float* parts = reinterpret_cast<float*>(smem_u);           // [warp][2][HP][ROW]
  uint32_t* prefix = smem_u + W * 2 * HP * ROW;              // batch + 1
  int32_t* lens = reinterpret_cast<int32_t*>(prefix + a.batch + 1);
  // of the warps' shares: their pass, and what the pass is
  struct Share {
    int b, hq0, heads;
    uint32_t first, units;  // the pass's units
  };
  // of the first and the last pass of this CTA, where they cross its ends
  struct Cross {
    uint32_t pass, c0, c1;  // its first and last CTA
    int last;               // whether this CTA arrived last
  };
  __shared__ uint32_t scan[W], longest[W], pass_of[2 * W], leader_of[2 * W];
  __shared__ Share share_of[2 * W];
  __shared__ Cross cross[2];
  __shared__ float4 group_stats[2 * W][HP];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, c = lane & 3;
  pdl_launch_dependents();
  if (threadIdx.x < 2 * W) pass_of[threadIdx.x] = kAtNone;
  pdl_wait();

  // ---- lengths and prefix sums of the sequences' units
  const uint32_t per_seq = static_cast<uint32_t>(a.hk * a.hgroups);
  auto units_of = [](int len) { return static_cast<uint32_t>((len + kAtKeys - 1) / kAtKeys + kAtPassUnits); };
  uint32_t most = 0;  // units of a pass
  {
    uint32_t carry = 0;
    for (int b0 = 0; b0 < a.batch; b0 += THREADS) {
      const int b = b0 + static_cast<int>(threadIdx.x);
      uint32_t n = 0;
      if (b < a.batch) {
        const int len = min(max(a.lengths[b], 0), a.max_len);
        lens[b] = len;
        n = units_of(len) * per_seq;
        most = max(most, units_of(len));
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
      for (int w = 0; w < W; ++w) {
        before += w < warp ? scan[w] : 0u;
        all += scan[w];
      }
      if (b < a.batch) prefix[b] = before + x - n;
      carry += all;
      __syncthreads();
    }
    if (threadIdx.x == 0) prefix[a.batch] = carry;
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) longest[warp] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) most = max(most, longest[w]);
  }
  // (a unit for every warp at least, where there are that many in all; so no
  // run is empty, and every CTA between a pass's first and last takes part)
  const uint32_t total = prefix[a.batch], ctas = min(gridDim.x, max(total / W, 1u));
  auto run_start = [&](uint32_t cta) { return static_cast<uint32_t>(static_cast<uint64_t>(cta) * total / ctas); };
  auto owner = [&](uint32_t unit) {
    return static_cast<uint32_t>((static_cast<uint64_t>(unit + 1) * ctas - 1) / total);
  };
  uint32_t t0, t1;
  const uint32_t passes = static_cast<uint32_t>(a.batch) * per_seq;
  const int64_t spare = static_cast<int64_t>(a.each + (a.extra > 0 ? 1u : 0u)) * most - kAtWhole * W;
  if (spare * gridDim.x <= total) {
    // Passes that are few and short, or of about the same length: as many whole
    // ones to a CTA, so that no join goes past it, which takes 4 us.  (Cut and
    // whole: 5 sequences of up to 200 tokens 8.6 us and 6.5; 32 / 8 heads of 128:
    // 64 of 100 tokens 13.4 and 9.4, 24 of 200 12.4 and 8.3, 256 of 512 57 and
    // 53, 38 of 500, 8 / 4 heads, 10.2 both; where a CTA's whole passes are 6
    // units a warp above an even share, 64 of 2048, 54.5 and 56.1.)
    if (blockIdx.x >= min(passes, gridDim.x)) return;
    auto pass_start = [&](uint32_t cta) {
      const uint32_t pass = cta * a.each + min(cta, a.extra), seq = magic_div(pass, a.div_seq);
      return pass == passes ? total : prefix[seq] + (pass - seq * per_seq) * units_of(lens[seq]);
    };
    t0 = pass_start(blockIdx.x);
    t1 = pass_start(blockIdx.x + 1);
  } else {
    if (blockIdx.x >= ctas) return;
    t0 = run_start(blockIdx.x);
    t1 = run_start(blockIdx.x + 1);
  }
  const uint32_t s0 = t0 + static_cast<uint32_t>(static_cast<uint64_t>(t1 - t0) * warp / W);
  const uint32_t s1 = t0 + static_cast<uint32_t>(static_cast<uint64_t>(t1 - t0) * (warp + 1) / W);
  int b = 0;
  {
    int lo = 0, hi = a.batch - 1;  // the last sequence whose prefix is <= s0
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= s0) lo = mid; else hi = mid - 1;
    }
    b = lo;
  }
  auto put4 = [&](int seq, int head_at, int d, float4 acc, float lt, float Rt) {
    const float f = ex2f(Rt) / lt;
    uint16_t* dst = a.out + static_cast<int64_t>(seq) * a.os + static_cast<int64_t>(head_at) * D + d;
    if (lt == 0.0f)
      st_global_v2(dst, 0u, 0u);
    else
      st_global_v2(dst, pack_pair16<BF16>(acc.x * f, acc.y * f), pack_pair16<BF16>(acc.z * f, acc.w * f));
  };

  for (uint32_t t = s0; t < s1;) {
    while (t >= prefix[b + 1]) ++b;
    const int len = lens[b];
    const uint32_t units = units_of(len);
    const uint32_t hh = (t - prefix[b]) / units, in = t - prefix[b] - hh * units;
    const uint32_t stop = min(units, in + (s1 - t));  // the share: units [in, stop) of the pass
    const int h = static_cast<int>(hh) / a.hgroups, hg = static_cast<int>(hh) - h * a.hgroups;
    const int key1 = min(len, static_cast<int>(stop) * kAtKeys);
    const int heads = min(HP, a.group - hg * HP);  // of this pass
    const int hq0 = h * a.group + hg * HP;
    int key = static_cast<int>(in) * kAtKeys;

    // ---- the first keys on their way
    uint4 kw[U][2][KP];
    uint32_t vw[U][4][VW];
    int kx[U][2], vx[U][2];
    auto page_of = [&](int at) -> uint32_t {
      if (at >= key1) return kAtNone;
      return static_cast<uint32_t>(
          a.table[static_cast<int64_t>(b) * a.table_stride + magic_div(static_cast<uint32_t>(at), a.div_page)]);
    };
    auto row_of = [&](int at, uint32_t page) -> int64_t {
      const int off = at - static_cast<int>(magic_div(static_cast<uint32_t>(at), a.div_page)) * a.page;
      return (static_cast<int64_t>(page) * a.hk + h) * a.page + off;
    };
    auto load_k = [&](int u, int at, uint32_t page) {
      if (page >= a.pages) return;
      const int64_t row = row_of(at, page);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int p = 0; p < KP; ++p) kw[u][i][p] = ld_stream_v4(a.k + (row + r + 8 * i) * D + p * 64 + c * 16);
        kx[u][i] = a.ke[row + r + 8 * i];
      }
    };
    auto load_v = [&](int u, int at, uint32_t page) {
      if (page >= a.pages) return;
      const int64_t row = row_of(at, page);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* p = a.v + (row + 2 * c + (i & 1) + 8 * (i >> 1)) * D + r * (D / 8);
        if constexpr (D == 128) {
          const uint4 x = ld_stream_v4(p);
          vw[u][i][0] = x.x; vw[u][i][1] = x.y; vw[u][i][2] = x.z; vw[u][i][3] = x.w;
        } else {
          const uint2 x = ld_stream_v2(p);
          vw[u][i][0] = x.x; vw[u][i][1] = x.y;
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) vx[u][i] = a.ve[row + r + 8 * i];
    };
    uint32_t page[U], next_page[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      page[u] = page_of(key + u * kAtKeys);
      next_page[u] = page_of(key + (U + u) * kAtKeys);
      load_k(u, key + u * kAtKeys, page[u]);
      load_v(u, key + u * kAtKeys, page[u]);
    }

    // ---- the queries as B fragments: lane (r, c) has head r's values
    // p*64 + c*16 + 4j + {0, 1 | 2, 3} for step (p, j), in fp16 (bf16 ones
    // times a power of two that brings the head's largest to [1, 4))
    uint32_t qf[KP * 4][2];
    float qscale[2];
    {
      uint4 w[KP][2];
#pragma unroll
      for (int p = 0; p < KP; ++p)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          w[p][e] = make_uint4(0u, 0u, 0u, 0u);
          if (r < heads)
            w[p][e] = *reinterpret_cast<const uint4*>(a.q + static_cast<int64_t>(b) * a.qs +
                                                      static_cast<int64_t>(hq0 + r) * D + p * 64 + c * 16 + e * 8);
        }
      float mine = a.cs, inv = 1.0f;
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
        // (at most 126: 2^-127 is none of pow2i's)
        const int e = min(max(static_cast<int>(top), 1) - 127, 126);
        inv = pow2i(-e);
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
            qf[p * 4 + j][0] = pack_pair16<false>(x0.x * inv, x0.y * inv);
            qf[p * 4 + j][1] = pack_pair16<false>(x1.x * inv, x1.y * inv);
          } else {
            qf[p * 4 + j][0] = w0;
            qf[p * 4 + j][1] = w1;
          }
        }
      // this lane's columns of S are heads 2c and 2c + 1
      qscale[0] = __shfl_sync(0xffffffffu, mine, 8 * c);
      qscale[1] = __shfl_sync(0xffffffffu, mine, 8 * c + 4);
    }

    const bool large = __any_sync(0xffffffffu, qscale[0] >= 2.0f || qscale[1] >= 2.0f);  // (keys' powers end at 2^127)

    float o[MT][4];
    float l[2] = {0.0f, 0.0f}, m[2] = {-INFINITY, -INFINITY}, R[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < MT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;

    // ---- the keys
    for (; key < key1; key += U * kAtKeys) {
      const int next = key + U * kAtKeys;
      uint32_t page2[U];
      int valid[U];  // keys of the block (a page that is none holds none)
      float s[U][4], ve[U][2];
      bool over = false;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        page2[u] = page_of(next + (U + u) * kAtKeys);
        valid[u] = page[u] < a.pages ? min(16, max(key1 - key - u * kAtKeys, 0)) : 0;
        s[u][0] = s[u][1] = s[u][2] = s[u][3] = 0.0f;
#pragma unroll
        for (int p = 0; p < KP; ++p) {
          const uint32_t x0[4] = {kw[u][0][p].x, kw[u][0][p].y, kw[u][0][p].z, kw[u][0][p].w};
          const uint32_t x1[4] = {kw[u][1][p].x, kw[u][1][p].y, kw[u][1][p].z, kw[u][1][p].w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_16816(s[u], widen_lo(x0[j]), widen_lo(x1[j]), widen_hi(x0[j]), widen_hi(x1[j]), qf[p * 4 + j][0],
                      qf[p * 4 + j][1]);
        }
        const float f0 = key_power(kx[u][0]), f1 = key_power(kx[u][1]);
        ve[u][0] = static_cast<float>(vx[u][0] - 127);
        ve[u][1] = static_cast<float>(vx[u][1] - 127);
        load_k(u, next + u * kAtKeys, next_page[u]);
        // (the key's power with the query's first: they cancel where one is very
        // large and the other very small, and the sum times the former alone may
        // be past fp32.  Where they are both so large that their product is, a sum
        // of 0 stays 0.  At head_dim 128 that is asked for once a pass: 1 x 65536
        // tokens 30.4 us, always 30.75; at 64 it is always done: 16 x 4096 21.9 us,
        // asked for 22.3.)
        float g[4] = {f0 * qscale[0], f0 * qscale[1], f1 * qscale[0], f1 * qscale[1]};
        if (D == 64 || large) {
#pragma unroll
          for (int e = 0; e < 4; ++e) g[e] = fminf(g[e], FLT_MAX);
        }
        s[u][0] = r < valid[u] ? s[u][0] * g[0] : -INFINITY;
        s[u][1] = r < valid[u] ? s[u][1] * g[1] : -INFINITY;
        s[u][2] = r + 8 < valid[u] ? s[u][2] * g[2] : -INFINITY;
        s[u][3] = r + 8 < valid[u] ? s[u][3] * g[3] : -INFINITY;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float ref = m[e] == -INFINITY ? 0.0f : m[e];
          const float d0 = s[u][e] - ref, d1 = s[u][2 + e] - ref, top = R[e] + kAtLazy;
          over |= d0 > kAtLazy || d1 > kAtLazy || d0 + ve[u][0] > top || d1 + ve[u][1] > top;
        }
      }
      if (__any_sync(0xffffffffu, over)) {
        // move the references to these keys' maxima, where they are larger
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = -INFINITY, y = -INFINITY;
#pragma unroll
          for (int u = 0; u < U; ++u) x = fmaxf(x, fmaxf(s[u][e], s[u][2 + e]));
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, sh));
          const float mn = fmaxf(m[e], x), ref = mn == -INFINITY ? 0.0f : mn;
#pragma unroll
          for (int u = 0; u < U; ++u) y = fmaxf(y, fmaxf(s[u][e] - ref + ve[u][0], s[u][2 + e] - ref + ve[u][1]));
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, sh));
          const float moved = m[e] == -INFINITY ? -INFINITY : m[e] - ref;  // <= 0
          const float old = m[e] == -INFINITY ? -INFINITY : R[e] + moved;  // R against the new m
          const float Rn = fmaxf(rintf(old), ceilf(y));
          const float fl = ex2f(moved), fo = m[e] == -INFINITY ? 0.0f : ex2f(old - Rn);
          l[e] *= fl;
          m[e] = mn;
          R[e] = Rn;
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            o[i][e] *= fo;
            o[i][2 + e] *= fo;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float ref = m[e] == -INFINITY ? 0.0f : m[e];
          const float p0 = ex2f(s[u][e] - ref), p1 = ex2f(s[u][2 + e] - ref);
          l[e] += p0 + p1;
          // (R never set: every p is 0 or not a number)
          const float down = m[e] == -INFINITY ? 0.0f : R[e];
          w[e] = p0 * pow2i(static_cast<int>(ve[u][0] - down));
          w[2 + e] = p1 * pow2i(static_cast<int>(ve[u][1] - down));
        }
        const uint32_t b0 = transpose_8x8(pack_pair16<false>(w[0], w[1]));
        const uint32_t b1 = transpose_8x8(pack_pair16<false>(w[2], w[3]));
        if (valid[u] < 16) {  // what lies past the end may be anything, a NaN too
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (2 * c + (i & 1) + 8 * (i >> 1) >= valid[u]) {
#pragma unroll
              for (int j = 0; j < VW; ++j) vw[u][i][j] = 0u;
            }
        }
#pragma unroll
        for (int j = 0; j < VW; ++j) {
          const uint32_t lo0 = prmt(vw[u][0][j], vw[u][1][j], 0x5140u), lo1 = prmt(vw[u][0][j], vw[u][1][j], 0x7362u);
          const uint32_t hi0 = prmt(vw[u][2][j], vw[u][3][j], 0x5140u), hi1 = prmt(vw[u][2][j], vw[u][3][j], 0x7362u);
          mma_16816(o[2 * j], widen_lo(lo0), widen_hi(lo0), widen_lo(hi0), widen_hi(hi0), b0, b1);
          mma_16816(o[2 * j + 1], widen_lo(lo1), widen_hi(lo1), widen_lo(hi1), widen_hi(hi1), b0, b1);
        }
        load_v(u, next + u * kAtKeys, next_page[u]);
        page[u] = next_page[u];
        next_page[u] = page2[u];
      }
    }

    // ---- a whole pass to the output, a share to shared memory
    const bool whole = in == 0 && stop == units;
    const int part = warp * 2 + (t == s0 ? 0 : 1);
    if (!whole && lane == 0) {
      pass_of[part] = static_cast<uint32_t>(b) * per_seq + hh;
      share_of[part] = Share{b, hq0, heads, prefix[b] + hh * units, units};
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int sh = 4; sh < 32; sh <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], sh);
      const int head = 2 * c + e;
      if (head < heads) {
        float* row = parts + (part * HP + head) * ROW;
#pragma unroll
        for (int i = 0; i < MT; i += 2) {
          const float4 x = make_float4(o[i][e], o[i][2 + e], o[i + 1][e], o[i + 1][2 + e]);
          const int d = r * (D / 8) + 2 * i;
          if (whole)
            put4(b, hq0 + head, d, x, l[e], R[e]);
          else
            *reinterpret_cast<float4*>(row + d) = x;
        }
        if (!whole && r == 0) *reinterpret_cast<float4*>(row + D) = make_float4(l[e], m[e], R[e], 0.0f);
      }
    }
    t += stop - in;
  }
  __syncthreads();

  // ---- the warps' shares together: neighbouring ones of the same pass
  const uint32_t mine = pass_of[lane];
  const uint32_t used = __ballot_sync(0xffffffffu, mine != kAtNone);
  if (used == 0) return;
  const uint32_t below = used & ((1u << lane) - 1u);
  const uint32_t previous = __shfl_sync(0xffffffffu, mine, below ? 31 - __clz(below) : 0);
  const bool leads = mine != kAtNone && (!below || previous != mine);
  const uint32_t leaders = __ballot_sync(0xffffffffu, leads);
  // the places of the shares of place e's pass
  auto first_of = [&](uint32_t e) { return 31 - __clz((leaders | 1u) & ((2u << e) - 1u)); };
  auto end_of = [&](uint32_t e) {
    const uint32_t later = leaders & ~((2u << e) - 1u);
    return later ? __ffs(later) - 2 : 31;
  };
  if (warp == 0 && leads) leader_of[__popc(leaders & ((1u << lane) - 1u))] = lane;
  if (warp == W - 1 && lane < 2) {
    const uint32_t e = lane == 0 ? __ffs(used) - 1 : 31 - __clz(used);
    const Share x = share_of[e];
    Cross k{kAtNone, 0, 0, 0};
    if ((x.first < t0 || x.first + x.units > t1) && !(lane == 1 && (leaders & (leaders - 1)) == 0))
      k = Cross{pass_of[e], owner(x.first), owner(x.first + x.units - 1), 0};
    cross[lane] = k;
  }
  // the factors of the shares and their passes' {l, m, R}: a head a warp, a
  // share a lane
  if (const int head = warp; head < HP) {
    float4 st = make_float4(0.0f, -INFINITY, -INFINITY, 0.0f);
    float* row = parts + (lane * HP + head) * ROW + D;
    const bool has = mine != kAtNone && head < share_of[lane].heads;
    if (has) st = *reinterpret_cast<const float4*>(row);
    st = join_lanes(st.x, st.y, st.z, first_of(lane), end_of(lane));
    if (has) row[3] = st.w;
    if (leads) group_stats[lane][head] = st;
  }
  __syncthreads();
  constexpr int kItems = HP * (D / 4);
  for (int i = threadIdx.x; i < __popc(leaders) * kItems; i += THREADS) {
    const uint32_t e0 = leader_of[i / kItems];
    const int head = i % kItems / (D / 4), d = i % (D / 4) * 4;
    const Share x = share_of[e0];
    if (head >= x.heads) continue;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const uint32_t end = end_of(e0);
#pragma unroll 4
    for (uint32_t e = e0; e <= end; ++e) {
      if (!((used >> e) & 1u)) continue;
      const float* row = parts + (e * HP + head) * ROW;
      const float4 y = *reinterpret_cast<const float4*>(row + d);
      const float f = row[D + 3];
      acc.x += y.x * f;
      acc.y += y.y * f;
      acc.z += y.z * f;
      acc.w += y.w * f;
    }
    const float4 g = group_stats[e0][head];
    if (x.first >= t0 && x.first + x.units <= t1) {
      put4(x.b, x.hq0 + head, d, acc, g.x, g.z);
    } else {
      // (the pass's first CTA leaves its share in its second place: the first
      // place may be that of a pass that ends in it)
      float* row = a.part + ((static_cast<int64_t>(blockIdx.x) * 2 + (x.first >= t0 ? 1 : 0)) * HP + head) * ROW;
      *reinterpret_cast<float4*>(row + d) = acc;
      if (d == 0) *reinterpret_cast<float4*>(row + D) = g;
    }
  }
  if (cross[0].pass == kAtNone && cross[1].pass == kAtNone) return;

  // ---- the CTAs' shares, in two steps where there are many: kAtJoin
  // neighbours by the last of them to arrive, then those by the last of all
  __syncthreads();
  int32_t* const part_counters = a.counters + static_cast<int64_t>(a.batch) * per_seq;
  if (threadIdx.x < 2) {
    Cross& k = cross[threadIdx.x];
    if (k.pass != kAtNone) {
      const uint32_t n = k.c1 - k.c0 + 1, lo = (blockIdx.x - k.c0) / kAtJoin * kAtJoin;
      k.last = arrive_last(n <= kAtJoin ? a.counters + k.pass : part_counters + (k.c0 + lo) * 2 + (lo == 0 ? 1 : 0),
                           min(kAtJoin, n - lo));
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    const Cross k = cross[i];
    if (!k.last) continue;
    const Share x = share_of[i == 0 ? __ffs(used) - 1 : 31 - __clz(used)];
    const uint32_t n = k.c1 - k.c0 + 1, lo = (blockIdx.x - k.c0) / kAtJoin * kAtJoin;
    const bool all = n <= kAtJoin;
    auto slot_of = [&](uint32_t p) { return static_cast<int64_t>(k.c0 + p) * 2 + (p == 0 ? 1 : 0); };
    auto put = [&](int head, int d, float4 acc, float4 g) { put4(x.b, x.hq0 + head, d, acc, g.x, g.z); };
    join_parts<D>(a.part, parts, min(kAtJoin, n - lo), [&](uint32_t p) { return slot_of(lo + p); }, x.heads,
                           [&](int head, int d, float4 acc, float4 g) {
                             if (all) {
                               put(head, d, acc, g);
                             } else {
                               float* row = a.part + (slot_of(lo) * HP + head) * ROW;
                               *reinterpret_cast<float4*>(row + d) = acc;
                               if (d == 0) *reinterpret_cast<float4*>(row + D) = g;
                             }
                           });
    if (all) continue;
    const uint32_t groups = (n + kAtJoin - 1) / kAtJoin;
    if (threadIdx.x == 0) cross[i].last = arrive_last(a.counters + k.pass, groups);
    __syncthreads();
    if (cross[i].last)
      join_parts<D>(a.part, parts, groups, [&](uint32_t p) { return slot_of(p * kAtJoin); }, x.heads, put);
  }
}

struct AttendPlan {
  int hgroups, ctas;
  size_t part_bytes, bytes;
};

bool plan_attend(int32_t q_heads, int32_t k_heads, int32_t batch, AttendPlan* p) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  p->hgroups = (q_heads / k_heads + kAtHeads - 1) / kAtHeads;
  p->ctas = sms;
  // (room for the parts of any head_dim, so that the counters, which every run
  // leaves zero, are at the same place whatever else a workspace is used for)
  p->part_bytes = static_cast<size_t>(p->ctas) * 2 * kAtHeads * (kAtMaxDim + 4) * sizeof(float);
  p->bytes = p->part_bytes + (static_cast<size_t>(batch) * k_heads * p->hgroups + 2 * p->ctas) * sizeof(int32_t);
  return true;
}

template <int D, bool BF16>
cudaError_t launch_attend(const AttendArgs& a, int ctas, cudaStream_t stream) {
  constexpr size_t parts = sizeof(float) * kAtWarps * 2 * kAtHeads * (D + 4);
  constexpr size_t most = parts + sizeof(uint32_t) * (2 * kAtMaxBatch + 1);
  static_assert(most <= 227 * 1024 - 6 * 1024, "shared memory, with the 5 KiB that are not dynamic");
  const cudaError_t e = set_smem_once<cache_attend_kernel<D, BF16>>(static_cast<int>(most));
  if (e != cudaSuccess) return e;
  return launch_pdl(cache_attend_kernel<D, BF16>, dim3(static_cast<unsigned>(ctas)), dim3(kAtThreads),
                    parts + sizeof(uint32_t) * (2 * static_cast<size_t>(a.batch) + 1), stream, a);
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
  if (!lgt::plan_attend(q_heads, k_heads, batch, &p)) return GEMM_ERR_CUDA;
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
  // (units are counted in 32 bits, keys in 31)
  const int64_t max_len = static_cast<int64_t>(max_pages) * c.page_size;
  if (batch > lgt::kAtMaxBatch || max_len > (int64_t{1} << 30)) return GEMM_ERR_UNSUPPORTED;
  lgt::AttendPlan p;
  if (!lgt::plan_attend(q_heads, c.k_heads, batch, &p)) return GEMM_ERR_CUDA;
  const int64_t passes = static_cast<int64_t>(batch) * c.k_heads * p.hgroups;
  if ((max_len / lgt::kAtKeys + lgt::kAtPassUnits + 1) * passes >= (int64_t{1} << 31)) return GEMM_ERR_UNSUPPORTED;
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
  a.div_seq = lgt::magic_encode(static_cast<uint32_t>(a.hk * a.hgroups));
  a.each = static_cast<uint32_t>(std::max<int64_t>(passes / p.ctas, 1));
  a.extra = passes > p.ctas ? static_cast<uint32_t>(passes % p.ctas) : 0u;
  a.cs = (scale > 0.0f ? scale : 1.0f / std::sqrt(static_cast<float>(c.head_dim))) * 1.4426950408889634f;
  a.page = c.page_size;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = dtype == GEMM_BF16;
  cudaError_t e;
  if (c.head_dim == 128)
    e = bf16 ? lgt::launch_attend<128, true>(a, p.ctas, s) : lgt::launch_attend<128, false>(a, p.ctas, s);
  else
    e = bf16 ? lgt::launch_attend<64, true>(a, p.ctas, s) : lgt::launch_attend<64, false>(a, p.ctas, s);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  return GEMM_OK;
}
