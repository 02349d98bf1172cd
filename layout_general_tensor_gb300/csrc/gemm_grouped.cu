// Products over groups of rows (include/gemm_grouped.h) on tcgen05.
//
// Both forms are one kernel.  The matrix instruction's M side (128 rows of
// tensor-memory lanes a CTA, 256 a pair) takes C's contiguous index n, its N
// side C's row index, so a tile's accumulator is C transposed:
//   groups along M: M side = B of the group (n), N side = rows of A,  K = k
//   groups along K: M side = B's columns (n),    N side = A's columns, K = rows
// The rows of a group are thus on the side that the instruction takes in steps
// of 16 (32 a pair): a group of any size costs its own rows, rounded up, and not
// a tile's 128 (4 rows of 1536 x 2048: one eighth).  A group's rows are spread
// evenly over as few tiles as hold them.  Columns of the accumulator that stand
// for rows of another group are computed and not stored; they touch no other.
//
// Bound, and measured on one GB300 (copies run at 6.79 TB/s, library products at
// 1922 TFLOP/s, 1708 for long): with many rows a group the tensor pipe, and in runs
// of many such products the power limit (16384 rows of 16 groups, 4096 x 4096:
// 302 to 316 us alone, 1740 to 1820 TFLOP/s, pipe busy for 92 % of the time; 365 one after the
// other; along K, 2048 x 4096: 164 and 181); with few rows the weights' bytes (512
// rows of 128 groups, 1536 x 2048: 114 us, 97 % of the copy's rate; 8 rows of 8
// groups, 2048 x 4096: 20 us, of which 4 are its ends), along K with few rows
// the results' way out of tensor memory (1001 rows of 40 groups, 1000 x 2880: 52 us, of
// which 2 are the release of cleared rows to a pair; 23 without any results, 45 without
// copies to C, which alone would take 37); between the two, rounds of tiles (4000 rows of
// 24 groups, 3000 x 2880: 86 us, 68 by its bytes).
//
// Work.  The sizes are on the device, so every CTA sums them up itself (a scan
// over the groups' tiles in shared memory) and takes every G-th tile, G the
// CTAs or pairs: no launch depends on a size.  Within a group the tiles of one
// stretch of n follow each other, so that they read its weights together, in bands of
// eight of them, so that those that run at once have no more of the rows between them
// than the L2 holds (16384 rows of one group, 4096 x 4096: 391 us without, 335).  (Groups
// with the largest tiles first would leave small ones for the last round, but
// few rows and many weights then meet at the end: 4000 rows of 24 groups, 3000 x
// 2880, 85 to 88 us, and 16384 rows of 16 groups no better.)
//
// Where the tiles are too few for the SMs, the 2 to 8 CTAs of a cluster take a stretch
// of K each (SPLIT): each leaves its fp32 sums in its shared memory, and each adds and
// stores a share of the columns, in the CTAs' order (6 rows of one group, 632 x
// 2048: 12.2 to 7.2 us; 3302 rows along K, 192 x 168: 19.6 to 10.9).
//
// Groups along K.  The product's steps are 16 rows deep; what is left of a group
// behind its last whole step shares a step with the next group's rows, and a zero
// on one side would not cancel an infinity on the other.  So those rows have a
// small buffer of their own (16 rows of both operands, two of them), loaded as the
// tile begins, in which a warp of each CTA that has nothing else to do clears the
// rows beyond, and the product takes that step last.  (Cleared in the last block
// of 64 on its way through the ring, each tile waited for it: 16 groups of 1000
// rows, 2048 x 4096, 207 us against 157 for groups of 1024.  More than two buffers
// make no difference.)
//
// Roles (448 threads; pairs: in both CTAs):
//   warp 0, 12  copies of the M side (a stage's first, third, ... and the others,
//               where it takes several: a thread is held for each, and with one
//               warp a side that was the pace of a block)
//   warp 10, 13 the same of the N side
//   warp 1      tensor memory; issues the products (the even CTA of a pair)
//   warps 2..9  results      warp 11  clears the last step's rows (along K)
#include <algorithm>
#include <cstdint>
#include <cstdlib>
#include <new>

#include "gemm_grouped.h"
#include "group_tiles.h"
#include "groups.cuh"
#include "half_types.cuh"
#include "kernels.h"
#include "plan.h"
#include "ptx.cuh"

namespace lgt {
namespace {

constexpr int kGgThreads = 448;
constexpr int kGgEpiWarp0 = 2;
constexpr int kGgEpiWarps = 8;
constexpr int kGgQWarp = kGgEpiWarp0 + kGgEpiWarps;
constexpr int kGgClearWarp = kGgQWarp + 1;
constexpr int kGgOddP = kGgClearWarp + 1;  // (the N side's: the one behind it)
constexpr int kGgMaxGroups = 1024;
constexpr uint32_t kGgRows = 128;                       // M-side rows a CTA
constexpr uint32_t kGgPBytes = kGgRows * TILE_K * 2;    // 16 KiB of them a stage
constexpr uint32_t kGgChunk = 64 * TILE_K * 2;          // a box of 64 x 64 values along n or m
constexpr uint32_t kGgMost = 256;                       // N-side columns of a tile
// Rows of A in a copy: a tile's are as many copies as it has rows for, since a tile
// much narrower than the widest is the usual one (5266 rows of 69 groups, 3976 x
// 1144: 128 us with copies of 64 rows, 123 of 32, against 186 with one for the widest).
// From 512 rows a group on most tiles are wide (16384 rows of 16 groups, 4096 x 4096,
// one after the other: 377 us with copies of 32, 365 of 128; 20000 of 12, 2048 x 2048,
// 109 and 102; 6915 of 21, 4240 x 2008: 127 of 32, 133 of 64).
// Up to 4, one of half the size does for most (8 rows of 8 groups, 2048 x 4096, where
// each SM's stream is the limit: 24.1 us, 21.0).
constexpr uint32_t kGgPiece = 32;
constexpr int64_t kGgNarrowMean = 4;
constexpr int64_t kGgWideMean = 512;
constexpr uint32_t kGgMaxStages = 12;
constexpr uint32_t kGgEpiBytes = 2 * 2 * 8192;          // 32 rows of C, 128 values each, of two sets of warps, twice
constexpr uint32_t kGgStep = 16 * 128;                  // a step's 16 rows of 64 values along n or m
constexpr uint32_t kGgMaxSplit = 8;                     // CTAs that share a tile's K
constexpr uint32_t kGgRests = 2;                        // buffers for what is left behind a group's last whole step
constexpr uint32_t kGgBars = 2 * kGgMaxStages + 3 * kGgRests + 5;  // full, empty; rest landed, cleared, empty; accumulators full, empty; end
constexpr uint32_t kGgSmem = 227 * 1024;
constexpr uint64_t kGgSettleNs = 200ull * 1000ull * 1000ull;

struct GroupedArgs {
  CUtensorMap tm_p, tm_q;
  CUtensorMap tm_pr, tm_qr;  // along K: boxes of one step
  CUtensorMap tm_c;          // boxes of 32 rows of 64 values
  uint16_t* c;
  const int32_t* offsets;
  DeviceStatus* status;
  uint64_t wait_limit_ns;
  int64_t ldc, c_stride;
  int32_t groups, rows;
  int32_t along_k;
  int32_t n, m;           // extent of the M side; of the N side (along K)
  int32_t kb_total;       // blocks of K (along M)
  uint32_t p_tiles;
  uint32_t q_most;            // along M: rows of a tile at most
  uint32_t q_tiles, q_width;  // along K
  uint32_t q_box;             // columns of an N-side copy
  uint32_t q_chunks;          // along K: stretches of 64 columns, of each CTA
  uint32_t p_boxes, q_boxes;  // copies of a stage's operand
  int32_t p_whole, q_whole;   // the one copy is of several stretches
  uint32_t q_step;            // along K: what a tile's columns are a multiple of, a power of two
  uint32_t lg_most;           // along M: of q_most
  uint32_t recip[kGgBand + 1];  // band_reciprocals
  uint32_t stages, stage_bytes;
  uint32_t split;  // CTAs that share a tile's K (SPLIT)
  int32_t p_mn;
  uint32_t idesc;  // without N
  int32_t withhold;
};

// One tile.
struct GroupedTile {
  int32_t group;
  int32_t p0, q0;     // its first n; its first column of the N side (along M: a row of A)
  uint32_t count;     // columns to store
  uint32_t cols;      // of the product
  int32_t row0;       // along K: the group's first row
  int32_t steps;      // of the product, of 16
  int32_t nkb;        // blocks of 64 that hold them
  int32_t kb0;        // the first of them
  int32_t rest;       // along K: rows behind them
};

template <bool PAIR>
struct GroupedCfg {
  static constexpr uint32_t CTAS = PAIR ? 2 : 1;
  static constexpr uint32_t STEP = PAIR ? 32 : 16;  // of the product's N
};

template <bool PAIR, bool SPLIT>
struct GroupedWork {
  const uint32_t *off, *first;
  uint32_t tile, step, end;
  // along K: of the next tile, and of a step
  uint32_t g, r, step_g, step_r;
  __device__ GroupedWork(const GroupedArgs& a, const uint32_t* off_, const uint32_t* first_) : off(off_), first(first_) {
    const uint32_t ctas = SPLIT ? a.split : GroupedCfg<PAIR>::CTAS;
    tile = blockIdx.x / ctas;
    step = gridDim.x / ctas;
    end = a.along_k ? static_cast<uint32_t>(a.groups) * a.p_tiles * a.q_tiles : first[a.groups];
    if (a.along_k) {
      const uint32_t all = a.p_tiles * a.q_tiles;
      g = tile / all;
      r = tile - g * all;
      step_g = step / all;
      step_r = step - step_g * all;
    }
  }
  // (Every role asks for every tile, and short tiles take little longer than this did
  // with divisions: 1001 rows of 40 groups along K, 57.5 to 50.1 us.  There is one left
  // where a group has more than a band.)
  __device__ bool next(const GroupedArgs& a, GroupedTile& t) {
    if (tile >= end) return false;
    constexpr uint32_t STEP = GroupedCfg<PAIR>::STEP;
    const uint32_t u = tile;
    tile += step;
    if (a.along_k) {
      uint32_t p, q;
      tile_in_bands(a.recip, r, a.p_tiles, a.q_tiles, p, q);
      t.group = static_cast<int32_t>(g);
      t.p0 = static_cast<int32_t>(p * kGgRows * GroupedCfg<PAIR>::CTAS);
      const uint32_t q0 = q * a.q_width, len = off[g + 1] - off[g];
      t.q0 = static_cast<int32_t>(q0);
      t.count = min(a.q_width, static_cast<uint32_t>(a.m) - q0);
      t.cols = (t.count + a.q_step - 1) & ~(a.q_step - 1);
      t.row0 = static_cast<int32_t>(off[g]);
      t.steps = static_cast<int32_t>(len >> 4);
      t.rest = static_cast<int32_t>(len & 15u);
      g += step_g;
      r += step_r;
      if (r >= a.p_tiles * a.q_tiles) {
        r -= a.p_tiles * a.q_tiles;
        ++g;
      }
    } else {
      const uint32_t g = group_of(first, a.groups, u);
      const uint32_t len = off[g + 1] - off[g], tiles = (len + a.q_most - 1) >> a.lg_most;
      const uint32_t width = even_width(a.recip, len, tiles, STEP);
      uint32_t p, q;
      tile_in_bands(a.recip, u - first[g], a.p_tiles, tiles, p, q);
      t.group = static_cast<int32_t>(g);
      t.p0 = static_cast<int32_t>(p * kGgRows * GroupedCfg<PAIR>::CTAS);
      t.q0 = static_cast<int32_t>(off[g] + q * width);
      t.count = min(width, len - q * width);
      t.cols = (t.count + STEP - 1) / STEP * STEP;
      t.steps = a.kb_total * (TILE_K / 16);  // (the last block's end is zeros)
      t.rest = 0;
    }
    t.nkb = (t.steps + TILE_K / 16 - 1) / (TILE_K / 16);
    t.kb0 = 0;
    if constexpr (SPLIT) {
      // this CTA's stretch; the last one has the rest, too
      const uint32_t r = cluster_ctarank();
      t.kb0 = static_cast<int32_t>(static_cast<int64_t>(t.nkb) * r / a.split);
      t.nkb = static_cast<int32_t>(static_cast<int64_t>(t.nkb) * (r + 1) / a.split) - t.kb0;
      t.steps = min(t.steps - t.kb0 * (TILE_K / 16), t.nkb * (TILE_K / 16));
      if (r + 1 < a.split) t.rest = 0;
    }
    return true;
  }
};

template <bool PAIR, bool SPLIT, bool BF16>
__global__ void __launch_bounds__(kGgThreads, 1) grouped_kernel(const __grid_constant__ GroupedArgs a) {
  pdl_launch_dependents();
  constexpr uint32_t CTAS = GroupedCfg<PAIR>::CTAS;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw_base);
  const uint32_t rest_off = a.stages * a.stage_bytes;
  const uint32_t rest_bytes = a.along_k ? (2 + a.q_chunks) * kGgStep : 0u;  // each
  const uint32_t epi_off = rest_off + kGgRests * rest_bytes;
  const uint32_t bar0 = base + epi_off + kGgEpiBytes;
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + epi_off + kGgEpiBytes + kGgBars * 8);
  volatile uint32_t* tmem_slot = misc;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  uint32_t* off = misc + 36;  // (32 words of the scan's lie between)
  uint32_t* first = off + a.groups + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  auto full = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty = [&](uint32_t s) { return bar0 + 8u * (kGgMaxStages + s); };
  auto landed = [&](uint32_t b) { return bar0 + 8u * (2 * kGgMaxStages + b); };
  auto cleared = [&](uint32_t b) { return bar0 + 8u * (2 * kGgMaxStages + kGgRests + b); };
  auto rest_empty = [&](uint32_t b) { return bar0 + 8u * (2 * kGgMaxStages + 2 * kGgRests + b); };
  const uint32_t acc0 = bar0 + 8u * (2 * kGgMaxStages + 3 * kGgRests);
  auto accf = [&](int b) { return acc0 + 8u * b; };
  auto acce = [&](int b) { return acc0 + 16u + 8u * b; };
  const uint32_t end_bar = acc0 + 32u;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    const bool got = PAIR ? mbar_wait_bounded_cluster_sleep(bar, parity, a.wait_limit_ns, abort_flag)
                          : mbar_wait_bounded(bar, parity, a.wait_limit_ns, abort_flag);
    if (!got) {
      *abort_flag = 1;
      a.status->where = warp;
      a.status->code = GEMM_ERR_TIMEOUT;
    }
    return got;
  };
  // (for a whole warp: one lane looks; the others' accesses are ordered behind it by the
  // warp's barrier, which a shuffle is not)
  auto warp_wait = [&](uint32_t bar, uint32_t parity) {
    int got = 0;
    if (lane == 0) got = wait(bar, parity);
    __syncwarp();
    return __shfl_sync(0xffffffffu, got, 0) != 0;
  };

  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < a.stages; ++s) {
      mbar_init(full(s), 2);      // the two copying warps (of the even CTA), and the bytes
      mbar_init(empty(s), 1);     // the products' commit, to both CTAs
    }
    for (uint32_t b = 0; b < kGgRests; ++b) {
      mbar_init(landed(b), 2);      // the two copying warps of this CTA, and its bytes
      mbar_init(cleared(b), CTAS);  // the clearing warps
      mbar_init(rest_empty(b), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf(b), 1);
      mbar_init(acce(b), kGgEpiWarps * CTAS);
    }
    mbar_init(end_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&a.tm_p);
    tma_prefetch_desc(&a.tm_q);
    tma_prefetch_desc(&a.tm_c);
    if (a.along_k) {
      tma_prefetch_desc(&a.tm_pr);
      tma_prefetch_desc(&a.tm_qr);
    }
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(smem_u32(const_cast<uint32_t*>(tmem_slot)), 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), 512);
      tmem_relinquish();
    }
  }
  pdl_wait();  // (the operands, the offsets and C may be the previous kernel's)
  group_rows<kGgThreads>(a.offsets, a.groups, a.rows, off, misc + 4);
  __syncthreads();
  if (!a.along_k)
    group_tiles<kGgThreads>(
        a.groups, [&](uint32_t g) { return (off[g + 1] - off[g] + a.q_most - 1) / a.q_most * a.p_tiles; }, first, misc + 20);
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // the even CTA's barriers
  const uint32_t full_lead = PAIR ? mapa_shared(full(0), 0) : full(0);
  const uint32_t cleared_lead = PAIR ? mapa_shared(cleared(0), 0) : cleared(0);
  const uint32_t acce_lead = PAIR ? mapa_shared(acce(0), 0) : acce(0);

  GroupedWork<PAIR, SPLIT> work(a, off, first);
  GroupedTile t;
  if (warp == 0 || warp == kGgQWarp || warp >= kGgOddP) {
    // ------------------------------------------------------------ copies
    const bool is_p = warp == 0 || warp == kGgOddP, odd = warp >= kGgOddP;
    // (A second warp has a copy in every stage or in none: one that waited for stages
    // without would be bound to nobody, and could miss that a stage was used twice.)
    const uint32_t every = !is_p && !a.along_k ? 1u : 2u;
    if ((!odd || (every > 1 && (is_p ? a.p_boxes : a.q_boxes) > 1)) && elect_one()) {
      const CUtensorMap* tm = is_p ? &a.tm_p : &a.tm_q;
      const CUtensorMap* tm_rest = is_p ? &a.tm_pr : &a.tm_qr;
      const uint32_t at = is_p ? 0u : kGgPBytes;
      const uint32_t chunks = is_p ? 2u : a.q_chunks;
      const uint32_t box = is_p ? 64u : a.q_box;
      uint32_t bytes = is_p ? kGgPBytes : a.q_chunks * kGgChunk, boxes = is_p ? a.p_boxes : a.q_boxes;
      // coordinates: whether the box runs along K first; whether it is all of the stage's stretches
      const bool k_first = is_p ? !a.p_mn : !a.along_k, whole = is_p ? a.p_whole : a.q_whole;
      auto copy = [&](const CUtensorMap* map, uint32_t dst, uint32_t apart, uint32_t bar, int32_t x0, int32_t k, int32_t z) {
        const int32_t stretch = whole ? x0 >> 6 : 0;
        for (uint32_t j = odd; j < boxes; j += every) {
          const int32_t x = whole ? 0 : x0 + static_cast<int32_t>(box * j);
          if constexpr (PAIR)
            tma_load_4d_pair(dst + j * apart, map, bar, k_first ? k : x, k_first ? x : k, stretch, z);
          else
            tma_load_4d(dst + j * apart, map, bar, k_first ? k : x, k_first ? x : k, stretch, z);
        }
      };
      uint32_t s = 0, phase = 0, issued = 0, rests = 0;
      bool ok = true;
      while (ok && work.next(a, t)) {
        const int32_t x0 = is_p ? t.p0 + static_cast<int32_t>(rank * kGgRows)
                                : t.q0 + static_cast<int32_t>(rank * (t.cols / CTAS));
        const int32_t z = is_p && !a.along_k ? t.group : 0;
        if (!is_p && !a.along_k) {  // (as many rows as the tile has)
          boxes = (t.cols / CTAS + box - 1) / box;
          bytes = boxes * box * (TILE_K * 2);
        }
        const int32_t k0 = (a.along_k ? t.row0 : 0) + t.kb0 * TILE_K;
        if (t.rest > 0) {
          const uint32_t b = rests % kGgRests;
          if (!(ok = wait(rest_empty(b), (rests / kGgRests & 1u) ^ 1u))) break;
          if (!odd) mbar_arrive_expect_tx(landed(b), chunks * kGgStep);
          copy(tm_rest, base + rest_off + b * rest_bytes + (is_p ? 0u : 2 * kGgStep), kGgStep,
               PAIR ? mapa_shared(landed(b), rank) : landed(b), x0, k0 + t.steps * 16, z);
          ++rests;
        }
        for (int kb = 0; kb < t.nkb; ++kb) {
          if (!(ok = wait(empty(s), phase ^ 1u))) break;
          if (leader && !odd) mbar_arrive_expect_tx(full(s), bytes * CTAS);
          if (!(a.withhold && !is_p && blockIdx.x == 0 && issued == 0))
            copy(tm, base + s * a.stage_bytes + at, box * (TILE_K * 2), full_lead + 8u * s, x0, k0 + kb * TILE_K, z);
          ++issued;
          if (++s == a.stages) {
            s = 0;
            phase ^= 1u;
          }
        }
      }
      // Every commit to this CTA's barriers has arrived before it leaves.
      for (uint32_t i = issued > a.stages ? issued - a.stages : 0u; ok && i < issued; ++i)
        ok = wait(empty(i % a.stages), i / a.stages & 1u);
      for (uint32_t i = rests > kGgRests ? rests - kGgRests : 0u; ok && i < rests; ++i)
        ok = wait(rest_empty(i % kGgRests), i / kGgRests & 1u);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    // (the elected thread's operands go through uniform registers; descriptors are
    // one sum each, since this thread's own instructions are the pace)
    if (leader && elect_one()) {
      const uint32_t p_step = (a.p_mn ? 2048u : 32u) >> 4, q_step = (a.along_k ? 2048u : 32u) >> 4;
      const uint64_t p_desc = sw128_desc(base, a.p_mn ? kGgChunk : 16u, 1024u);
      const uint64_t q_desc = sw128_desc(base + kGgPBytes, a.along_k ? kGgChunk : 16u, 1024u);
      const uint32_t stage_step = a.stage_bytes >> 4;
      auto product = [](uint32_t d, uint64_t p, uint64_t q, uint32_t idesc, uint32_t accumulate) {
        if constexpr (PAIR)
          tc_mma_f16_ss_pair(d, p, q, idesc, accumulate);
        else
          tc_mma_f16_ss(d, p, q, idesc, accumulate);
      };
      uint32_t s = 0, phase = 0, uses = 0, rests = 0;
      bool ok = true;
      while (ok && work.next(a, t)) {
        if (t.nkb == 0 && t.rest == 0) continue;
        const int buf = static_cast<int>(uses & 1u);
        if (!(ok = wait(acce(buf), (uses >> 1 & 1u) ^ 1u))) break;
        tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(buf) * kGgMost;
        const uint32_t idesc = a.idesc | (t.cols >> 3) << 17;
        for (int kb = 0; kb < t.nkb; ++kb) {
          if (!(ok = wait(full(s), phase))) break;
          tc_fence_after();
          const uint64_t pd = p_desc + s * stage_step, qd = q_desc + s * stage_step;
          const int here = t.steps - kb * (TILE_K / 16);
#pragma unroll
          for (int k = 0; k < TILE_K / 16; ++k) {
            if (k >= here) break;
            product(d, pd + k * p_step, qd + k * q_step, idesc, (kb | k) != 0 ? 1u : 0u);
          }
          if constexpr (PAIR)
            tc_commit_pair_mc(empty(s), 0x3);
          else
            tc_commit(empty(s));
          if (++s == a.stages) {
            s = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (t.rest > 0) {
          const uint32_t b = rests % kGgRests;
          if (!(ok = wait(cleared(b), rests / kGgRests & 1u))) break;
          tc_fence_after();
          const uint32_t at = base + rest_off + b * rest_bytes;
          product(d, sw128_desc(at, kGgStep, 1024u), sw128_desc(at + 2 * kGgStep, kGgStep, 1024u), idesc, t.nkb > 0 ? 1u : 0u);
          if constexpr (PAIR)
            tc_commit_pair_mc(rest_empty(b), 0x3);
          else
            tc_commit(rest_empty(b));
          ++rests;
        }
        if constexpr (PAIR)
          tc_commit_pair_mc(accf(buf), 0x3);
        else
          tc_commit(accf(buf));
        ++uses;
      }
      if constexpr (PAIR)
        tc_commit_pair_mc(end_bar, 0x1);
      else
        tc_commit(end_bar);
    }
  } else if (warp == kGgClearWarp) {
    // ------------------------------------------------------------ rows of the next group
    if (a.along_k) {
      uint32_t rests = 0;
      bool ok = true;
      while (ok && work.next(a, t)) {
        if (t.rest == 0) continue;
        const uint32_t b = rests % kGgRests;
        if (!(ok = warp_wait(landed(b), rests / kGgRests & 1u))) break;
        ++rests;
        const uint32_t at = base + rest_off + b * rest_bytes;
        for (uint32_t c = 0; c < 2 + a.q_chunks; ++c)
          for (uint32_t i = static_cast<uint32_t>(t.rest) * 128u + lane * 16u; i < kGgStep; i += 512u)
            st_shared_v4(at + c * kGgStep + i, 0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
        // (A pair's product is the even CTA's: the zeros are released to the cluster, which
        // costs 1 us before the last step; 17024 rows of 121 groups, 376 x 6584, 187 to 199 us.)
        if (lane == 0) {
          if constexpr (PAIR)
            mbar_arrive_cluster(cleared_lead + 8u * b);
          else
            mbar_arrive(cleared(b));
        }
      }
    }
  } else {
    // ------------------------------------------------------------ results
    // Two warps of a set (each has a quarter of the lanes) put 32 columns of 64 values
    // together in shared memory, and a copy of the box takes them to C (by single stores
    // of 256 bytes in a piece, four warps together, 1001 rows of 40 groups along K,
    // 1000 x 2880, took 61.8 us, so 57.5; of 64 bytes, a warp's own, 127 rows of 41,
    // 920 x 7928, 217 against 177).  The arrivals at the even CTA release nothing, since
    // tensor memory is all that they speak of: released to the cluster they wait for the
    // stores, 2000 to 3500 cycles of a tile's 6500 (1001 rows of 40 groups 52 us against
    // 76, 127 of 41 128 against 192, 32768 of 8 with K = 256 and 4096 columns 69 against 96).
    const uint32_t quad = static_cast<uint32_t>(warp & 3), set = static_cast<uint32_t>(warp - kGgEpiWarp0) / 4;
    const uint32_t half = quad >> 1, stage = base + epi_off + set * 2 * 8192u + half * 4096u;
    // Places as a copy of boxes takes them: row r at 128 r, its 16-byte pieces exchanged
    // so that eight rows' pieces are in eight different bank groups.
    const uint32_t put = stage + (lane & 7u) * 128u + (((quad & 1u) * 4u + static_cast<uint32_t>(lane >> 3)) ^ (lane & 7u)) * 16u;
    const uint32_t row = (quad & 1u) * 16u + static_cast<uint32_t>(lane >> 3), piece = static_cast<uint32_t>(lane & 7);
    const bool issues = (quad & 1u) == 0 && lane == 0;
    uint32_t uses = 0, pieces = 0;
    while (work.next(a, t)) {
      const int buf = static_cast<int>(uses & 1u);
      const bool some = t.nkb > 0 || t.rest > 0;
      if (some) {
        // (the warps meet below, so they give up together)
        if (named_bar_or(2 + set * 2 + half, 64, !warp_wait(accf(buf), uses >> 1 & 1u))) break;
        tc_fence_after();
      }
      const uint32_t d = tmem + static_cast<uint32_t>(buf) * kGgMost + (quad * 32u << 16);
      if constexpr (SPLIT) {
        // this CTA's sums, column by column, where the ring was (it has but this tile)
        for (uint32_t c = set * 32; c < t.count; c += 64) {
          uint32_t v[32];
          if (some) {
            tc_ld_32x32b_x32(d + c, v);
            tc_wait_ld_regs(v);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0u;
          }
#pragma unroll
          for (uint32_t i = 0; i < 32; ++i)
            st_shared_f32(base + (c + i) * (kGgRows * 4) + (quad * 32u + lane) * 4u, __uint_as_float(v[i]));
        }
        break;
      }
      const int32_t n0 = t.p0 + static_cast<int32_t>(rank * kGgRows + half * 64u), n = n0 + static_cast<int32_t>(piece * 8u);
      uint16_t* out = a.c + (a.along_k ? t.group * a.c_stride : 0) + static_cast<int64_t>(t.q0) * a.ldc + n;
      const bool last = a.along_k && t.q0 + static_cast<int32_t>(t.count) == a.m;  // (rows behind the matrix are not stored)
      // (the sets take turns of 32 columns; the next ones are on their way while these are stored)
      uint32_t x[16], y[16];
      auto load = [&](uint32_t c) {
        tc_ld_16x256b_x4(d + c, x);
        tc_ld_16x256b_x4(d + c + (16u << 16), y);
      };
      // the accumulators are free as soon as they have been read, long before the results are stored
      auto done = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR)
            mbar_arrive_tmem_read(acce_lead + 8u * buf);
          else
            mbar_arrive(acce(buf));
        }
      };
      if (!some) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = y[i] = 0u;
      } else if (set * 32 < t.count) {
        load(set * 32);
      } else {
        done();
      }
      for (uint32_t c = set * 32; c < t.count; c += 64, ++pieces) {
        if (some) {
          tc_wait_ld_regs(x);
          tc_regs_after_wait(y);
        }
        uint32_t w[16];
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
          w[4 * i] = pack_pair16<BF16>(__uint_as_float(x[4 * i]), __uint_as_float(x[4 * i + 1]));
          w[4 * i + 1] = pack_pair16<BF16>(__uint_as_float(x[4 * i + 2]), __uint_as_float(x[4 * i + 3]));
          w[4 * i + 2] = pack_pair16<BF16>(__uint_as_float(y[4 * i]), __uint_as_float(y[4 * i + 1]));
          w[4 * i + 3] = pack_pair16<BF16>(__uint_as_float(y[4 * i + 2]), __uint_as_float(y[4 * i + 3]));
        }
        if (some) {
          if (c + 64 < t.count)
            load(c + 64);
          else
            done();
        }
        // (of two places, the one that was read before the two warps last met)
        const uint32_t here = (pieces & 1u) * 8192u;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i)
          stmatrix_x4_trans(put + here + i * 1024u, w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        fence_proxy_async_smem();
        if (issues) bulk_wait_group_read<0>();  // (the other place)
        named_bar_sync(2 + set * 2 + half, 64);
        // A box that has rows of another tile goes by single stores.
        if (c + 32 <= t.count || last) {
          if (issues && n0 < a.n) {
            tma_store_4d(&a.tm_c, stage + here, n0, t.q0 + static_cast<int32_t>(c), 0, a.along_k ? t.group : 0);
            bulk_commit_group();
          }
        } else {
#pragma unroll
          for (uint32_t i = 0; i < 4; ++i) {
            const uint32_t r = row + 4 * i;
            const uint4 v = ld_shared_v4(stage + here + r * 128u + ((piece ^ (r & 7u)) << 4));
            if (c + r < t.count && n < a.n) st_global_v4(out + static_cast<int64_t>(c + r) * a.ldc, v.x, v.y, v.z, v.w);
          }
        }
      }
      uses += some;
    }
    if (issues) bulk_wait_group<0>();
  }

  // ------------------------------------------------------------ end
  __syncthreads();
  if (*abort_flag) {
    // Copies that were made may still be landing, on a barrier that will not
    // complete: they take microseconds, and are given far more.
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < kGgSettleNs) {
    }
  }
  if (leader && warp == 1) {
    volatile int no_abort = 0;
    mbar_wait_bounded(end_bar, 0, drain_ns(a.wait_limit_ns), &no_abort);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR || SPLIT) cluster_sync_all();
  tc_fence_after();
  if constexpr (SPLIT) {
    // A share of the columns, the CTAs' sums in order: a column a warp, four values a lane.
    GroupedWork<PAIR, SPLIT> again(a, off, first);
    if (again.next(a, t)) {
      const uint32_t r = cluster_ctarank(), c1 = t.count * (r + 1) / a.split;
      const int32_t n = t.p0 + 4 * lane;
      for (uint32_t c = t.count * r / a.split + warp; c < c1; c += kGgThreads / 32) {
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (uint32_t i = 0; i < a.split; ++i) {
          const float4 v = ld_cluster_f32x4(mapa_shared(base + c * (kGgRows * 4) + lane * 16u, i));
          sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
        }
        if (n < a.n)
          st_global_v2(a.c + (a.along_k ? t.group * a.c_stride : 0) + (t.q0 + static_cast<int64_t>(c)) * a.ldc + n,
                       pack_pair16<BF16>(sum.x, sum.y), pack_pair16<BF16>(sum.z, sum.w));
      }
    }
    cluster_sync_all();  // (the others have read this CTA's)
  }
  if (warp == 1) {
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem, 512);
    else
      tmem_dealloc(tmem, 512);
  }
}

template <bool PAIR, bool SPLIT, bool BF16>
cudaError_t launch_grouped_as(const GroupedArgs& a, unsigned workers, cudaStream_t stream) {
  const cudaError_t e = set_smem_once<grouped_kernel<PAIR, SPLIT, BF16>>(static_cast<int>(kGgSmem));
  if (e != cudaSuccess) return e;
  const unsigned ctas = PAIR ? 2 : SPLIT ? a.split : 1;
  if (ctas > 1)
    return launch_pdl_cluster(grouped_kernel<PAIR, SPLIT, BF16>, dim3(ctas * workers), dim3(kGgThreads), kGgSmem, stream, ctas, a);
  return launch_pdl(grouped_kernel<PAIR, SPLIT, BF16>, dim3(workers), dim3(kGgThreads), kGgSmem, stream, a);
}

template <bool BF16>
cudaError_t launch_grouped(const GroupedArgs& a, bool pair, unsigned workers, cudaStream_t stream) {
  return pair          ? launch_grouped_as<true, false, BF16>(a, workers, stream)
         : a.split > 1 ? launch_grouped_as<false, true, BF16>(a, workers, stream)
                       : launch_grouped_as<false, false, BF16>(a, workers, stream);
}

// Clusters of `ctas` CTAs of the split form that run at once on this device; below 0: an error.
template <bool BF16>
int resident_split_clusters(unsigned ctas) {
  constexpr auto kernel = grouped_kernel<false, true, BF16>;
  if (set_smem_once<kernel>(static_cast<int>(kGgSmem)) != cudaSuccess) return -1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kGgThreads);
  cfg.dynamicSmemBytes = kGgSmem;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  return cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg) == cudaSuccess ? clusters : -1;
}

// A matrix [d2][d1][d0] with pitches s1 and s2 in elements, by boxes of 64 of d0
// times box1 of d1.  `stretches` > 1 of them, next to each other along d0, are one
// box, one after the other in shared memory: d0 in pieces of 64 is a dimension of
// its own then (d0 has to be a multiple of 64, or the last piece of the last row
// would reach past the matrix).
bool encode_matrices(CUtensorMap* map, const void* ptr, bool bf16, int64_t d0, int64_t d1, int64_t d2, int64_t s1, int64_t s2,
                     uint32_t box1, uint32_t stretches) {
  auto enc = get_encoder();
  if (!enc) return false;
  const bool cut = stretches > 1;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(cut ? 64 : d0), static_cast<cuuint64_t>(d1), static_cast<cuuint64_t>(cut ? d0 / 64 : 1),
                        static_cast<cuuint64_t>(d2)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(s1) * 2, 128, static_cast<cuuint64_t>(s2) * 2};
  cuuint32_t box[4] = {64, box1, stretches, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(ptr), dims,
             strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

uint64_t grouped_wait_limit() {
  const char* s = std::getenv("LGT_GEMM_WAIT_LIMIT_MS");
  if (s && *s) {
    const double ms = std::atof(s);
    if (ms > 0) return static_cast<uint64_t>(ms * 1e6);
  }
  return 2000ull * 1000ull * 1000ull;  // 2 s
}

int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

}  // namespace
}  // namespace lgt

struct gemm_grouped_plan {
  gemm_grouped_desc_t d;
  int device = -1;
  int sms = 0;
  int resident[lgt::kGgMaxSplit + 1] = {};  // clusters of so many CTAs (SPLIT) that run at once
  lgt::DeviceStatus* d_status = nullptr;
  uint64_t wait_limit_ns = 0;
  int withhold_armed = 0;  // gemm_grouped_withhold_load: the next run withholds a load (one shot)
};

extern "C" {

gemm_status_t gemm_grouped_create(const gemm_grouped_desc_t* desc, gemm_grouped_plan_t** plan) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  *plan = nullptr;
  if (!desc) return GEMM_ERR_INVALID_ARG;
  const gemm_grouped_desc_t& d = *desc;
  auto size = [](int64_t v) { return v >= 8 && v % 8 == 0 && v < (int64_t{1} << 30); };
  const bool along_k = d.form == GEMM_GROUPED_K;
  if (d.groups < 1 || d.groups > lgt::kGgMaxGroups || (d.form != GEMM_GROUPED_M && !along_k) || !size(d.N) ||
      (d.dtype != GEMM_F16 && d.dtype != GEMM_BF16) ||
      (along_k ? !size(d.M) || d.K != 0 || d.b_layout != GEMM_MN_CONTIG
               : !size(d.K) || d.M != 0 || (d.b_layout != GEMM_K_CONTIG && d.b_layout != GEMM_MN_CONTIG)))
    return GEMM_ERR_INVALID_ARG;
  gemm_grouped_plan* p = new (std::nothrow) gemm_grouped_plan();
  if (!p) return GEMM_ERR_CUDA;
  p->d = d;
  p->wait_limit_ns = lgt::grouped_wait_limit();
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
  for (unsigned c = 2; p->device >= 0 && c <= lgt::kGgMaxSplit; ++c) {
    p->resident[c] = d.dtype == GEMM_BF16 ? lgt::resident_split_clusters<true>(c) : lgt::resident_split_clusters<false>(c);
    if (p->resident[c] < 0) {
      cudaGetLastError();
      cudaFree(p->d_status);
      delete p;
      return GEMM_ERR_CUDA;
    }
  }
  *plan = p;
  return GEMM_OK;
}

gemm_status_t gemm_grouped_run(gemm_grouped_plan_t* plan, const void* A, int64_t lda, const void* B, int64_t ldb,
                               int64_t b_stride, const int32_t* offsets, int64_t rows, void* C, int64_t ldc,
                               int64_t c_stride, void* stream) {
  using namespace lgt;
  if (!plan || rows < 0) return GEMM_ERR_INVALID_ARG;
  const gemm_grouped_desc_t& d = plan->d;
  const bool along_k = d.form == GEMM_GROUPED_K, b_mn = d.b_layout == GEMM_MN_CONTIG, bf16 = d.dtype == GEMM_BF16;
  const int64_t a_row = along_k ? d.M : d.K, b_row = b_mn ? d.N : d.K;
  if (lda == 0) lda = a_row;
  if (ldb == 0) ldb = b_row;
  if (ldc == 0) ldc = d.N;
  const int64_t b_rows = b_mn ? d.K : d.N;
  // (a copy's pitches are below 2^40 bytes, and no product of a pitch and a size passes 64 bits)
  constexpr int64_t kPitch = int64_t{1} << 32, kStride = int64_t{1} << 38;
  for (int64_t v : {lda, ldb, ldc})
    if (v < 0 || v % 8 != 0 || v > kPitch) return GEMM_ERR_INVALID_ARG;
  if (along_k)
    b_stride = 8;
  else
    c_stride = 0;
  if (!along_k && b_stride == 0) b_stride = b_rows * ldb;
  if (along_k && c_stride == 0) c_stride = d.M * ldc;
  for (int64_t v : {b_stride, c_stride})
    if (v < 0 || v % 8 != 0 || v > kStride) return GEMM_ERR_INVALID_ARG;
  if (lda < a_row || ldb < b_row || ldc < d.N || (!along_k && b_stride < (b_rows - 1) * ldb + b_row) ||
      (along_k && c_stride < (d.M - 1) * ldc + d.N))
    return GEMM_ERR_INVALID_ARG;
  if (rows == 0 && !along_k) return GEMM_OK;
  if (!offsets || !C || (rows > 0 && (!A || !B))) return GEMM_ERR_INVALID_ARG;
  for (const void* p : {A, B, static_cast<const void*>(C)})
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return GEMM_ERR_ALIGNMENT;
  if (reinterpret_cast<uintptr_t>(offsets) % 4 != 0) return GEMM_ERR_ALIGNMENT;
  if (rows > (int64_t{1} << 30)) return GEMM_ERR_UNSUPPORTED;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  if (dev != plan->device) return GEMM_ERR_INVALID_ARG;  // (the status word is there)

  GroupedArgs a = {};
  band_reciprocals(a.recip);
  const int64_t busy = std::min<int64_t>(d.groups, std::max<int64_t>(rows, 1));
  const int64_t mean = (rows + busy - 1) / busy;
  // Few rows a group: tiles as wide as twice the mean, so that most groups have one, and
  // the ring is deep (512 rows of 128 groups, 1536 x 2048: 124 us in tiles of 256), but
  // no narrower than 64 for the groups that have many (8192 rows in 4 of 512 groups,
  // 1024 x 2048: 104 us in tiles of 16 to 32, 58 of 64).
  const uint32_t narrow = 2 * mean <= 64 ? 64 : 2 * mean <= 128 ? 128 : kGgMost;
  // Tiles of single CTAs (along M a guess between their least and greatest number,
  // since the sizes are not known here), and blocks of K of each: where clusters for all of them
  // run at once, and the blocks that a CTA then does not do are worth the exchange (a
  // block 0.25 us, the exchange 2.5), K is split, over as many CTAs as that allows (428
  // rows of 4 groups, 952 x 5672: four 19.5 us, two 28, none 33.7; 3881 of 10, 2176 x
  // 920, 340 tiles: none 24.6, two 66).
  const int64_t single = (along_k ? static_cast<int64_t>(d.groups) * ((d.M + kGgMost - 1) / kGgMost)
                                  : std::min(rows / narrow + busy, std::max(busy + busy / 8, rows / narrow + (busy + 3) / 2))) *
                         ((d.N + kGgRows - 1) / kGgRows);
  const int64_t deep = (along_k ? mean : d.K) / TILE_K;
  a.split = 1;
  for (uint32_t c = 2; c <= kGgMaxSplit; ++c)
    if (single <= plan->resident[c] && deep * (c - 1) >= 10 * c) a.split = c;
  // A pair reads each row of A for 256 columns, single CTAs with tiles of fitting width
  // keep more of the weights on their way (64 groups, 2048 x 2048, of 100 rows: 103 us
  // single, 96 paired; of 64: 95, 93; of 24: 85, 89).
  const bool pair = a.split == 1 && d.N > kGgRows && (along_k ? d.M > 64 : mean > 56);
  const uint32_t ctas = pair ? 2 : 1, step = pair ? 32 : 16;
  a.p_tiles = static_cast<uint32_t>((d.N + kGgRows * ctas - 1) / (kGgRows * ctas));
  int64_t tiles;
  // Operands that run along n or m: one copy a stage where the matrix is whole
  // stretches of 64 (the copying thread is held for each: 4096 x 4096 of [k][n], 16
  // groups of 1024 rows, 293 us against 356 with one warp a side), else one a stretch.
  const bool p_whole = b_mn && d.N % 64 == 0, q_whole = along_k && d.M % 64 == 0;
  a.p_boxes = b_mn && !p_whole ? 2 : 1;
  a.q_boxes = 1;
  a.q_step = q_whole ? 64 * ctas : step;
  if (along_k) {
    a.q_tiles = static_cast<uint32_t>((d.M + kGgMost - 1) / kGgMost);
    a.q_width = static_cast<uint32_t>(up((d.M + a.q_tiles - 1) / a.q_tiles, a.q_step));
    a.q_chunks = (a.q_width / ctas + 63) / 64;
    if (!q_whole) a.q_boxes = a.q_chunks;
    a.q_box = 64;
    a.stage_bytes = kGgPBytes + a.q_chunks * kGgChunk;
    tiles = static_cast<int64_t>(d.groups) * a.p_tiles * a.q_tiles;
  } else {
    a.q_most = pair ? kGgMost : narrow;
    while (1u << a.lg_most < a.q_most) ++a.lg_most;
    a.q_box = mean >= kGgWideMean ? a.q_most / ctas : mean <= kGgNarrowMean ? kGgPiece / 2 : kGgPiece;
    a.stage_bytes = kGgPBytes + a.q_most / ctas * TILE_K * 2;
    tiles = (rows / a.q_most + busy) * a.p_tiles;
  }
  if (tiles >= (int64_t{1} << 31)) return GEMM_ERR_UNSUPPORTED;
  const uint32_t tables = 144 + static_cast<uint32_t>(d.groups + 1) * 8;
  const uint32_t rest = along_k ? kGgRests * (2 + a.q_chunks) * kGgStep : 0;
  a.stages = std::min<uint32_t>(kGgMaxStages, (kGgSmem - 1024 - kGgEpiBytes - kGgBars * 8 - tables - rest) / a.stage_bytes);

  // (no rows: nothing is copied, any valid address will do)
  const void* ap = rows > 0 ? A : C;
  const void* bp = rows > 0 ? B : C;
  const int64_t some = std::max<int64_t>(rows, 1);
  const uint32_t p_stretches = p_whole ? 2 : 1, q_stretches = q_whole ? a.q_chunks : 1;
  a.p_whole = p_stretches > 1;
  a.q_whole = q_stretches > 1;
  const bool encoded =
      along_k ? encode_matrices(&a.tm_p, bp, bf16, d.N, some, 1, ldb, ldb, 64, p_stretches) &&
                    encode_matrices(&a.tm_q, ap, bf16, d.M, some, 1, lda, lda, 64, q_stretches) &&
                    encode_matrices(&a.tm_pr, bp, bf16, d.N, some, 1, ldb, ldb, 16, p_stretches) &&
                    encode_matrices(&a.tm_qr, ap, bf16, d.M, some, 1, lda, lda, 16, q_stretches)
              : encode_matrices(&a.tm_p, bp, bf16, b_row, b_rows, d.groups, ldb, b_stride, b_mn ? 64 : kGgRows, p_stretches) &&
                    encode_matrices(&a.tm_q, ap, bf16, d.K, some, 1, lda, lda, a.q_box, 1);
  if (!encoded) return GEMM_ERR_CUDA;
  if (!encode_matrices(&a.tm_c, C, bf16, d.N, along_k ? d.M : rows, along_k ? d.groups : 1, ldc, along_k ? c_stride : ldc, 32, 1))
    return GEMM_ERR_CUDA;
  a.c = static_cast<uint16_t*>(C);
  a.offsets = offsets;
  a.status = plan->d_status;
  // (a wait may be for all of a tile's blocks)
  a.wait_limit_ns = plan->wait_limit_ns + static_cast<uint64_t>((along_k ? rows : d.K) / TILE_K) * 2000;
  a.ldc = ldc;
  a.c_stride = c_stride;
  a.groups = d.groups;
  a.rows = static_cast<int32_t>(rows);
  a.along_k = along_k;
  a.n = static_cast<int32_t>(d.N);
  a.m = static_cast<int32_t>(d.M);
  a.kb_total = static_cast<int32_t>((d.K + TILE_K - 1) / TILE_K);
  a.p_mn = b_mn;
  a.idesc = idesc_f16(bf16, b_mn, along_k, kGgRows * ctas, 0);
  a.withhold = plan->withhold_armed ? __atomic_exchange_n(&plan->withhold_armed, 0, __ATOMIC_ACQ_REL) : 0;
  // (split, every tile has a cluster of its own)
  const unsigned workers = static_cast<unsigned>(a.split > 1 ? tiles : std::min<int64_t>(tiles, plan->sms / ctas));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((bf16 ? launch_grouped<true>(a, pair, workers, s) : launch_grouped<false>(a, pair, workers, s)) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  return GEMM_OK;
}

gemm_status_t gemm_grouped_sync_status(gemm_grouped_plan_t* plan, void* stream) {
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

gemm_status_t gemm_grouped_withhold_load(gemm_grouped_plan_t* plan) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  __atomic_store_n(&plan->withhold_armed, 1, __ATOMIC_RELEASE);
  return GEMM_OK;
}

gemm_status_t gemm_grouped_destroy(gemm_grouped_plan_t* plan) {
  if (!plan) return GEMM_OK;
  if (plan->d_status) cudaFree(plan->d_status);
  delete plan;
  return GEMM_OK;
}

}  // extern "C"
