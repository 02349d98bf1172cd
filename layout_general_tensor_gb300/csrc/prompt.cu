// Attention over packed prompts, causal, with grouped heads
// (include/attn_prompt.h).
//
// Rows.  All `group` query heads of a key head share its keys, so a tile of
// the tensor core's 128 rows is T = 128 / group tokens times their group
// heads (row = token * group + head; the TMA box of Q is that shape, so the
// rows arrive in this order), and a short prompt or a single query with many
// heads still fills rows.  A CTA takes two tiles, 2T neighbouring tokens, and
// walks the keys that any of them sees in blocks of 128; blocks past the last
// visible key are not touched.
//
//   S = Q K^T      tcgen05, both operands K-major in 128-byte swizzled
//                  shared memory, fp32 in tensor memory.
//   P = 2^(s - m)  one row a thread, the 128 logits of a block in registers,
//                  so no maximum or sum crosses threads; m is a reference
//                  that is moved (and O rescaled) only when a block exceeds
//                  it by 2^8; P goes back to tensor memory in 16 bits.
//   O += P V       tcgen05, A = P from tensor memory, B = V as it lies
//                  (MN-major).
// The two tiles alternate: while the tensor core works on one tile's
// products, the other tile's softmax runs.
//
// Warps (384 threads): 0-3 softmax of tile 0, 4-7 of tile 1, 8 loads, 9 issues
// the products, 10 and 11 look over the rows of V that some query of the CTA
// must not see, since a weight of 0 does not cancel an infinity or a NaN: rows
// that no query sees (later ones, or the next sequence's) are cleared; in the
// others (2T at most) values that are not finite are, and are added to the
// results of the queries that do see them at the end, where a sum with a
// positive weight would have left the same.  Tensor memory: S of the tiles at columns 0 and 128, O at 256 and
// 256 + head_dim; P lies over its own S (head_dim 128: the columns are all
// taken; the products that read P and write the next S are of one shape and
// one issuing thread, which keeps them in order) or behind O (head_dim 64).
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <new>

#include "attn_prompt.h"
#include "half_types.cuh"
#include "kernels.h"
#include "plan.h"
#include "ptx.cuh"

namespace lgt {
namespace {

constexpr int kPrThreads = 384;
constexpr int kPrRows = 128;   // rows of a tile
constexpr int kPrKeys = 128;   // keys of a block
constexpr int kPrTimeout = GEMM_ERR_TIMEOUT;
constexpr float kPrLazy = 8.0f;

struct PromptArgs {
  CUtensorMap tm_q;        // {head_dim, q_heads, rows}, box {64, group, T}
  CUtensorMap tm_k, tm_v;  // {head_dim, k_heads, rows}, box {64, 1, 128}
  const uint16_t* v;
  uint16_t* out;
  const int32_t *cu_q, *cu_k;
  DeviceStatus* status;
  uint64_t wait_limit_ns;
  int64_t vs, os;
  int32_t batch, total_q, total_k;
  int32_t hk, group, tok;  // tok: T
  int32_t causal;
  MagicDiv div_hk, div_group, div_pair;  // div_pair: by 2T
  float cs;  // scale * log2(e)
  uint32_t idesc_s, idesc_pv;
};

template <int D>
struct PromptCfg {
  static constexpr uint32_t CHUNK = 128u * 128u;      // 64 values of 128 rows
  static constexpr uint32_t TILE = (D / 64) * CHUNK;  // a tile of Q, K or V
  static constexpr int NS = D == 128 ? 5 : 9;         // ring of K and V tiles, in the order they are used
  static constexpr uint32_t Q_OFF = 0;                // two tiles
  static constexpr uint32_t RING_OFF = 2 * TILE;
  static constexpr uint32_t BAR_OFF = RING_OFF + NS * TILE;
  // full[NS], empty[NS], q_full[2], s_full[2], p_full[2][2], o_full[2], v_go[3], v_clean[3], teardown
  static constexpr int NBARS = 2 * NS + 17;
  static constexpr uint32_t MISC_OFF = BAR_OFF + ((NBARS * 8 + 15) & ~15);
  static constexpr uint32_t SMEM = MISC_OFF + 16 + 1024;  // slack for the 1024-byte alignment
  static constexpr uint32_t S_COL = 128;                  // between the tiles' S
  static constexpr uint32_t O_COL = 256;
  static constexpr uint32_t P_COL = D == 128 ? 0 : 384;
  static constexpr uint32_t P_STEP = D == 128 ? 128 : 64;
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// Whether this lane is the one that issues for its (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t x, y, z, d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c.x), "f"(c.y));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t x, y, d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
  return r;
}

__device__ __forceinline__ void st_tmem_x32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void st_tmem_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void prompt_timeout(const PromptArgs& a, volatile int* abort_flag, int where) {
  *abort_flag = 1;
  if (atomicCAS(&a.status->code, 0, kPrTimeout) == 0) a.status->where = where;
}

// A bounded wait whose outcome is the whole warp's: a lane that gave up while
// another saw the phase complete would part from it at the next warp barrier.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, limit_ns, abort_flag));
}

// What a CTA works on: 2T tokens of one sequence and key head.
struct PromptUnit {
  int row0, tokens;     // first row of Q, tokens (1 .. 2T); 0: nothing
  int key_row, nk;      // first row of K and V, keys
  int shift;            // token i of the unit sees keys <= i + shift
};

// Unit `u` of the list (sequences in order, each one's last tokens -- the
// most keys -- first); every lane of the warp returns the same.
__device__ __forceinline__ PromptUnit find_unit(const PromptArgs& a, uint32_t u) {
  const int lane = threadIdx.x & 31;
  PromptUnit r{0, 0, 0, 0, 0};
  uint32_t before = 0;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    const int b = b0 + lane;
    int q0 = 0, nq = 0;
    if (b < a.batch) {
      q0 = min(max(a.cu_q[b], 0), a.total_q);
      nq = max(min(a.cu_q[b + 1], a.total_q) - q0, 0);
    }
    const uint32_t n = magic_div(static_cast<uint32_t>(nq) + 2u * a.tok - 1u, a.div_pair);
    uint32_t x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const uint32_t all = __shfl_sync(0xffffffffu, x, 31);
    if (u - before < all) {  // (u >= before)
      const uint32_t in = u - before;
      const unsigned hit = __ballot_sync(0xffffffffu, x > in);
      const int src = __ffs(hit) - 1;
      const int sq0 = __shfl_sync(0xffffffffu, q0, src), snq = __shfl_sync(0xffffffffu, nq, src);
      const uint32_t units = __shfl_sync(0xffffffffu, n, src), first = __shfl_sync(0xffffffffu, x - n, src);
      const int i0 = static_cast<int>(units - 1u - (in - first)) * 2 * a.tok;
      const int sb = b0 + src;
      const int k0 = min(max(a.cu_k[sb], 0), a.total_k);
      const int nk = max(min(a.cu_k[sb + 1], a.total_k) - k0, 0);
      r.row0 = sq0 + i0;
      r.tokens = min(2 * a.tok, snq - i0);
      r.key_row = k0;
      r.nk = nk;
      r.shift = i0 + nk - snq;
      return r;
    }
    before += all;
  }
  return r;
}

// The sign bit of each half of a word whose exponent is all ones.
template <bool BF16>
__device__ __forceinline__ uint32_t odd_halves(uint32_t w) {
  constexpr uint32_t kExp = BF16 ? 0x7f807f80u : 0x7c007c00u, kOne = BF16 ? 0x00800080u : 0x04000400u;
  return ((w & kExp) + kOne) & 0x80008000u;
}
// All bits of the halves whose sign bits are set.
__device__ __forceinline__ uint32_t spread_halves(uint32_t signs) { return (signs >> 15) * 0xffffu; }

// Add the values of keys [from, to) that are not finite, columns col and
// col + 1 of V, to a query's results.
template <bool BF16>
__device__ __forceinline__ void add_odd(const PromptArgs& a, int key_row, int from, int to, int col, float& lo, float& hi) {
  for (int k = from; k < to; ++k) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(a.v + static_cast<int64_t>(key_row + k) * a.vs + col);
    const uint32_t bad = odd_halves<BF16>(w);
    const float2 x = unpack_pair16<BF16>(w);
    if (bad & 0x8000u) lo += x.x;
    if (bad & 0x80000000u) hi += x.y;
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kPrThreads, 1) prompt_kernel(const __grid_constant__ PromptArgs a) {
  using C = PromptCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw_base);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

  const uint32_t bar0 = base + C::BAR_OFF;
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (C::NS + s); };
  auto q_full = [&](int t) { return bar0 + 8u * (2 * C::NS + t); };
  auto s_full = [&](int t) { return bar0 + 8u * (2 * C::NS + 2 + t); };
  auto p_full = [&](int t, int half) { return bar0 + 8u * (2 * C::NS + 4 + 2 * t + half); };
  auto o_full = [&](int t) { return bar0 + 8u * (2 * C::NS + 8 + t); };
  auto v_go = [&](int i) { return bar0 + 8u * (2 * C::NS + 10 + i); };
  auto v_clean = [&](int i) { return bar0 + 8u * (2 * C::NS + 13 + i); };
  const uint32_t teardown = bar0 + 8u * (2 * C::NS + 16);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
  volatile int* odd_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 8);  // V held values that are not finite

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(q_full(t), 1);
      mbar_init(s_full(t), 1);
      mbar_init(p_full(t, 0), 4);  // the tile's softmax warps
      mbar_init(p_full(t, 1), 4);
      mbar_init(o_full(t), 1);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(v_go(i), 1);
      mbar_init(v_clean(i), 2);  // both looking warps
    }
    mbar_init(teardown, 1);
    *abort_flag = 0;
    *odd_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&a.tm_q);
    tma_prefetch_desc(&a.tm_k);
    tma_prefetch_desc(&a.tm_v);
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();

  uint32_t unit, h;
  magic_divmod(blockIdx.x, a.div_hk, unit, h);
  const PromptUnit w = find_unit(a, unit);
  // tokens, visible keys and blocks of the two tiles
  int toks[2], blocks[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    toks[t] = min(max(w.tokens - t * a.tok, 0), a.tok);
    const int last = t * a.tok + toks[t] - 1;
    const int vis = toks[t] == 0 ? 0 : a.causal ? min(max(last + w.shift + 1, 0), w.nk) : w.nk;
    blocks[t] = (vis + kPrKeys - 1) / kPrKeys;
  }
  const int nb = max(blocks[0], blocks[1]);
  // keys that every token of the CTA sees, and that any does; the blocks from
  // `mixed` on (three at most: they span 2T keys) hold some that not all see
  const int all_see = a.causal ? min(max(w.shift + 1, 0), w.nk) : w.nk;
  const int any_sees = a.causal ? min(max(w.tokens + w.shift, 0), w.nk) : w.nk;
  const int mixed = all_see / kPrKeys;

  int issued = 0;  // loads of the ring that were issued (warp 8)
  bool q_issued = false;

  if (warp == 8) {
    // -------------------------------------------------------------- loads
    const bool leader = elect_one();
    bool ok = true;
    auto load_q = [&](int t) {
      if (!leader || blocks[t] == 0) return;
      mbar_arrive_expect_tx(q_full(t), static_cast<uint32_t>(a.tok * a.group) * 128u * (D / 64));
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        tma_load_3d(base + C::Q_OFF + t * C::TILE + c * C::CHUNK, &a.tm_q, q_full(t), c * 64,
                    static_cast<int32_t>(h) * a.group, w.row0 + t * a.tok);
    };
    load_q(0);
    for (int n = 0; ok && n < 2 * nb; ++n) {
      const int s = n % C::NS;
      if (n >= C::NS && !warp_wait(empty(s), ((n / C::NS) - 1) & 1, a.wait_limit_ns, abort_flag)) {
        ok = false;
        break;
      }
      if (leader) {
        mbar_arrive_expect_tx(full(s), C::TILE);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(base + C::RING_OFF + s * C::TILE + c * C::CHUNK, (n & 1) ? &a.tm_v : &a.tm_k, full(s), c * 64,
                      static_cast<int32_t>(h), w.key_row + (n >> 1) * kPrKeys);
      }
      __syncwarp();
      issued = n + 1;
      // (only now, so that the lookers wait for this load's phase and no earlier one)
      if ((n & 1) && (n >> 1) >= mixed && leader) mbar_arrive(v_go((n >> 1) - mixed));
      if (n == 0) load_q(1);
    }
    q_issued = true;
    if (!ok && lane == 0 && !*abort_flag) prompt_timeout(a, abort_flag, 0);
  } else if (warp == 9) {
    // ----------------------------------------------------------- products
    // One thread does it all.  The tensor core takes the products in the
    // order of their issue, so the order is the schedule: P V of a tile as
    // its halves of P come, then the tile's next S, then the other tile's.
    // Waits on loads stand before products that queue up anyway.
    if (elect_one()) {
      bool ok = true;
      auto wait = [&](uint32_t bar, uint32_t parity) {
        if (ok) ok = mbar_wait_bounded(bar, parity, a.wait_limit_ns, abort_flag);
        return ok;
      };
      auto wait_full = [&](int n) { return wait(full(n % C::NS), (n / C::NS) & 1); };
      auto issue_s = [&](int t, int n) {
        const uint32_t kb = base + C::RING_OFF + (n % C::NS) * C::TILE, qb = base + C::Q_OFF + t * C::TILE;
        // 16 values of d are 32 bytes further in a 64-value chunk
        const uint64_t qd = sw128_desc(qb, 16u, 1024u), kd = sw128_desc(kb, 16u, 1024u);
        const uint32_t dst = tmem + t * C::S_COL;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t off = ((k >> 2) * C::CHUNK + (k & 3) * 32u) >> 4;
          tc_mma_f16_ss(dst, qd + off, kd + off, a.idesc_s, k > 0 ? 1u : 0u);
        }
        tc_commit(s_full(t));
      };
      auto issue_pv = [&](int t, int n, int half, bool first) {
        const uint64_t vd = sw128_desc(base + C::RING_OFF + (n % C::NS) * C::TILE, C::CHUNK, 1024u);
        const uint32_t dst = tmem + C::O_COL + t * D, pa = tmem + C::P_COL + t * C::P_STEP;
        // 16 keys are 2 KiB of V and 8 columns of P
#pragma unroll
        for (int i = 0; i < kPrKeys / 32; ++i) {
          const uint32_t k = half * (kPrKeys / 32) + i;
          mma_ts(dst, pa + k * 8, vd + static_cast<uint64_t>(k * 2048u >> 4), a.idesc_pv, (first && i == 0) ? 0u : 1u);
        }
      };
      if (nb > 0 && wait_full(0)) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (blocks[t] > 0 && wait(q_full(t), 0)) {
            tc_fence_after();
            issue_s(t, 0);
          }
        if (ok) tc_commit(empty(0));
        wait_full(1);
      }
      for (int j = 0; ok && j < nb; ++j) {
        const int vn = 2 * j + 1, kn = 2 * j + 2;
        if (j >= mixed && !wait(v_clean(j - mixed), 0)) break;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (j < blocks[t]) {
            if (!wait(p_full(t, 0), j & 1)) break;
            tc_fence_after();
            issue_pv(t, vn, 0, j == 0);
            if (t == 0 && j + 1 < nb && !wait_full(kn)) break;
            if (!wait(p_full(t, 1), j & 1)) break;
            tc_fence_after();
            issue_pv(t, vn, 1, false);
            if (j + 1 == blocks[t]) tc_commit(o_full(t));
          } else if (t == 0 && j + 1 < nb && !wait_full(kn)) {
            break;
          }
          if (t == 1) tc_commit(empty(vn % C::NS));
          if (t == 1 && j + 1 < nb && !wait_full(vn + 2)) break;
          if (j + 1 < blocks[t]) issue_s(t, kn);
        }
        if (ok && j + 1 < nb) tc_commit(empty(kn % C::NS));
      }
      if (!ok && !*abort_flag) prompt_timeout(a, abort_flag, 1);
      tc_commit(teardown);  // every product is done before the tensor memory is freed
    }
    __syncwarp();
  } else if (warp >= 10) {
    // ------------------------------------------- rows of V that not all see
    for (int j = mixed; j < nb; ++j) {
      const int n = 2 * j + 1, s = n % C::NS;
      if (!warp_wait(v_go(j - mixed), 0, a.wait_limit_ns, abort_flag) ||
          !warp_wait(full(s), (n / C::NS) & 1, a.wait_limit_ns, abort_flag)) {
        if (lane == 0 && !*abort_flag) prompt_timeout(a, abort_flag, 3);
        break;
      }
      const uint32_t vb = base + C::RING_OFF + s * C::TILE;
      const int look = max(all_see - j * kPrKeys, 0), clear = min(any_sees - j * kPrKeys, kPrKeys);
      uint32_t odd = 0;
      for (int i = look * 8 + (warp - 10) * 32 + lane; i < clear * 8; i += 64) {
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const uint4 x = ld_shared_v4(vb + c * C::CHUNK + i * 16);
          const uint32_t y = odd_halves<BF16>(x.x) | odd_halves<BF16>(x.y) | odd_halves<BF16>(x.z) | odd_halves<BF16>(x.w);
          if (y) {
            odd = 1;
            st_shared_v4(vb + c * C::CHUNK + i * 16, x.x & ~spread_halves(odd_halves<BF16>(x.x)),
                         x.y & ~spread_halves(odd_halves<BF16>(x.y)), x.z & ~spread_halves(odd_halves<BF16>(x.z)),
                         x.w & ~spread_halves(odd_halves<BF16>(x.w)));
          }
        }
      }
      for (int i = clear * 8 + (warp - 10) * 32 + lane; i < kPrKeys * 8; i += 64)
#pragma unroll
        for (int c = 0; c < D / 64; ++c) st_shared_v4(vb + c * C::CHUNK + i * 16, 0u, 0u, 0u, 0u);
      if (odd) *odd_flag = 1;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_clean(j - mixed));
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;  // this warp's tensor-memory lanes
    const uint32_t s_addr = tmem + lanes + t * C::S_COL;
    const uint32_t p_addr = tmem + lanes + C::P_COL + t * C::P_STEP;
    const uint32_t o_addr = tmem + lanes + C::O_COL + t * D;
    uint32_t tok, g;
    magic_divmod(static_cast<uint32_t>(row), a.div_group, tok, g);
    const bool live = static_cast<int>(tok) < toks[t];
    const int vis = a.causal ? min(static_cast<int>(tok) + t * a.tok + w.shift + 1, w.nk) : w.nk;
    float m = -INFINITY, l = 0.0f;
    bool ok = true;
    const int my_blocks = blocks[t];
    for (int j = 0; j < my_blocks; ++j) {
      if (!warp_wait(s_full(t), j & 1, a.wait_limit_ns, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // The first half of P against the reference as it stands, while the
      // block's maximum is found; in the rare block that exceeds the
      // reference by 2^kPrLazy in some row (and the first), the reference
      // moves and the half is made again.
      const int valid = vis - j * kPrKeys;
      const bool masked = __any_sync(0xffffffffu, valid < kPrKeys);
      const float2 cs2 = make_float2(a.cs, a.cs);
      float2 sum[4];
      uint32_t sv[128], pk[32];
      while (true) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          tc_ld_32x32b_x32(s_addr + 32u * i, *reinterpret_cast<uint32_t(*)[32]>(sv + 32 * i));
        tc_wait_ld_regs(sv);
        if (masked) {
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i >= valid) sv[i] = __float_as_uint(-INFINITY);
        }
        // (a row that has seen no key keeps weights of 2^-inf = 0)
        const float ref = m == -INFINITY ? 0.0f : m;
        const float2 neg = make_float2(-ref, -ref);
        float mp[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          sum[u] = make_float2(0.0f, 0.0f);
          mp[u] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float2 x = fma2(make_float2(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1])), cs2, neg);
          const float2 e = make_float2(ex2(x.x), ex2(x.y));
          sum[i & 3] = add2(sum[i & 3], e);
          pk[i] = pack_pair16<BF16>(e.x, e.y);
          mp[i & 3] = max3(mp[i & 3], __uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1]));
          mp[i & 3] = max3(mp[i & 3], __uint_as_float(sv[64 + 2 * i]), __uint_as_float(sv[64 + 2 * i + 1]));
        }
        const float mx = fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3])) * a.cs;
        const bool over = mx > m + kPrLazy;
        if (!__any_sync(0xffffffffu, over)) break;
        const float alpha = over ? ex2(m - mx) : 1.0f;  // 0 at the first block with a visible key
        if (over) m = mx;
        l *= alpha;
        if (j > 0) {
          // the product before has completed: this S was issued after it by
          // the same thread, and its barrier covers all that was issued before
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t v[32];
            tc_ld_32x32b_x32(o_addr + c, v);
            tc_wait_ld_regs(v);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
            st_tmem_x32(o_addr + c, v);
          }
          st_tmem_wait();
        }
      }
      st_tmem_x32(p_addr, pk);
      st_tmem_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full(t, 0));
      const float ref = m == -INFINITY ? 0.0f : m;
      const float2 neg = make_float2(-ref, -ref);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float2 x = fma2(make_float2(__uint_as_float(sv[64 + 2 * i]), __uint_as_float(sv[64 + 2 * i + 1])), cs2, neg);
        const float2 e = make_float2(ex2(x.x), ex2(x.y));
        sum[i & 3] = add2(sum[i & 3], e);
        pk[i] = pack_pair16<BF16>(e.x, e.y);
      }
      st_tmem_x32(p_addr + 32u, pk);
      st_tmem_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full(t, 1));
      const float2 s4 = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
      l += s4.x + s4.y;
    }
    if (ok && my_blocks > 0) ok = warp_wait(o_full(t), 0, a.wait_limit_ns, abort_flag);
    if (ok) {
      tc_fence_after();
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const bool odd = *odd_flag != 0;  // (set before the last product was let go)
      uint16_t* dst = a.out + static_cast<int64_t>(w.row0 + t * a.tok + static_cast<int>(tok)) * a.os +
                      static_cast<int64_t>(h * a.group + g) * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t v[32];
        if (my_blocks > 0) {
          tc_ld_32x32b_x32(o_addr + c, v);
          tc_wait_ld_regs(v);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0u;
        }
        if (live) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float lo = __uint_as_float(v[8 * q + 2 * e]) * inv, hi = __uint_as_float(v[8 * q + 2 * e + 1]) * inv;
              if (odd) add_odd<BF16>(a, w.key_row, all_see, vis, static_cast<int>(h) * D + c + 8 * q + 2 * e, lo, hi);
              x[e] = l == 0.0f ? 0u : pack_pair16<BF16>(lo, hi);
            }
            st_global_v4(dst + c + 8 * q, x[0], x[1], x[2], x[3]);
          }
        }
      }
    } else if (lane == 0 && !*abort_flag) {
      prompt_timeout(a, abort_flag, 2);
    }
  }

  // ------------------------------------------------------------ teardown
  __syncthreads();
  if (warp == 8 && *abort_flag) {
    // let the loads still in flight land before the CTA exits
    volatile int no_abort = 0;
    if (q_issued)
      for (int t = 0; t < 2; ++t)
        if (blocks[t] > 0) mbar_wait_bounded(q_full(t), 0, a.wait_limit_ns, &no_abort);
    for (int n = issued > C::NS ? issued - C::NS : 0; n < issued; ++n)
      mbar_wait_bounded(full(n % C::NS), (n / C::NS) & 1, a.wait_limit_ns, &no_abort);
  }
  if (warp == 9) {
    volatile int no_abort = 0;
    mbar_wait_bounded(teardown, 0, a.wait_limit_ns, &no_abort);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

template <int D, bool BF16>
cudaError_t launch_prompt(const PromptArgs& a, unsigned grid, cudaStream_t stream) {
  using C = PromptCfg<D>;
  const cudaError_t e = set_smem_once<prompt_kernel<D, BF16>>(static_cast<int>(C::SMEM));
  if (e != cudaSuccess) return e;
  return launch_pdl(prompt_kernel<D, BF16>, dim3(grid), dim3(kPrThreads), C::SMEM, stream, a);
}

// Rows of `heads` heads, pitch `stride` elements: boxes of 64 values, `box_heads` heads, `box_rows` rows.
bool encode_rows(CUtensorMap* map, const void* ptr, int dtype, int64_t d, int64_t heads, int64_t rows, int64_t stride,
                 int box_heads, int box_rows) {
  auto enc = get_encoder();
  if (!enc) return false;
  const CUtensorMapDataType dt =
      dtype == GEMM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(stride) * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, dt, 3, const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

uint64_t prompt_wait_limit() {
  const char* s = std::getenv("LGT_GEMM_WAIT_LIMIT_MS");
  if (s && *s) {
    const double ms = std::atof(s);
    if (ms > 0) return static_cast<uint64_t>(ms * 1e6);
  }
  return 2000ull * 1000ull * 1000ull;  // 2 s
}

}  // namespace
}  // namespace lgt

struct attn_prompt_plan {
  attn_prompt_desc_t d;
  lgt::DeviceStatus* d_status = nullptr;
  uint64_t wait_limit_ns = 0;
};

extern "C" {

gemm_status_t attn_prompt_create(const attn_prompt_desc_t* desc, attn_prompt_plan_t** plan) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  *plan = nullptr;
  if (!desc) return GEMM_ERR_INVALID_ARG;
  const attn_prompt_desc_t& d = *desc;
  if (d.q_heads < 1 || d.k_heads < 1 || d.q_heads % d.k_heads != 0 || d.q_heads / d.k_heads > lgt::kPrRows ||
      (d.head_dim != 64 && d.head_dim != 128) || (d.dtype != GEMM_F16 && d.dtype != GEMM_BF16) ||
      (d.causal != 0 && d.causal != 1) || !(d.scale >= 0.0f) || std::isinf(d.scale))
    return GEMM_ERR_INVALID_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  attn_prompt_plan* p = new (std::nothrow) attn_prompt_plan();
  if (!p) return GEMM_ERR_CUDA;
  p->d = d;
  p->wait_limit_ns = lgt::prompt_wait_limit();
  if (cudaMalloc(&p->d_status, 16) != cudaSuccess || cudaMemset(p->d_status, 0, 16) != cudaSuccess) {
    cudaGetLastError();
    if (p->d_status) cudaFree(p->d_status);
    delete p;
    return GEMM_ERR_CUDA;
  }
  *plan = p;
  return GEMM_OK;
}

gemm_status_t attn_prompt_run(attn_prompt_plan_t* plan, const void* Q, int64_t q_stride, const void* K,
                              int64_t k_stride, const void* V, int64_t v_stride, const int32_t* cu_q,
                              const int32_t* cu_k, int32_t batch, int64_t total_q, int64_t total_k, void* out,
                              int64_t out_stride, void* stream) {
  if (!plan || batch < 0 || total_q < 0 || total_k < 0) return GEMM_ERR_INVALID_ARG;
  const attn_prompt_desc_t& d = plan->d;
  const int64_t qrow = static_cast<int64_t>(d.q_heads) * d.head_dim, krow = static_cast<int64_t>(d.k_heads) * d.head_dim;
  int64_t* strides[4] = {&q_stride, &out_stride, &k_stride, &v_stride};
  for (int i = 0; i < 4; ++i) {
    const int64_t row = i < 2 ? qrow : krow;
    if (*strides[i] == 0) *strides[i] = row;
    if (*strides[i] < row || *strides[i] % 8 != 0) return GEMM_ERR_INVALID_ARG;
  }
  if (batch == 0 || total_q == 0) return GEMM_OK;
  if (!Q || !out || !cu_q || !cu_k || (total_k > 0 && (!K || !V))) return GEMM_ERR_INVALID_ARG;
  for (const void* p : {Q, K, V, static_cast<const void*>(out)})
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return GEMM_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(cu_q) | reinterpret_cast<uintptr_t>(cu_k)) % 4 != 0) return GEMM_ERR_ALIGNMENT;
  const int group = d.q_heads / d.k_heads, tok = lgt::kPrRows / group;
  // a sequence of n tokens has at most n / 2T + 1 units
  const int64_t units = (total_q / (2 * tok) + batch) * d.k_heads;
  if (total_q > (int64_t{1} << 30) || total_k > (int64_t{1} << 30) || units >= (int64_t{1} << 31))
    return GEMM_ERR_UNSUPPORTED;
  lgt::PromptArgs a;
  // (no keys: nothing is loaded, any valid address will do)
  const void* kp = total_k > 0 ? K : Q;
  const void* vp = total_k > 0 ? V : Q;
  if (!lgt::encode_rows(&a.tm_q, Q, d.dtype, d.head_dim, d.q_heads, total_q, q_stride, group, tok) ||
      !lgt::encode_rows(&a.tm_k, kp, d.dtype, d.head_dim, d.k_heads, total_k > 0 ? total_k : 1, k_stride, 1, lgt::kPrKeys) ||
      !lgt::encode_rows(&a.tm_v, vp, d.dtype, d.head_dim, d.k_heads, total_k > 0 ? total_k : 1, v_stride, 1, lgt::kPrKeys))
    return GEMM_ERR_CUDA;
  a.v = static_cast<const uint16_t*>(V);
  a.vs = v_stride;
  a.out = static_cast<uint16_t*>(out);
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.status = plan->d_status;
  a.wait_limit_ns = plan->wait_limit_ns;
  a.os = out_stride;
  a.batch = batch;
  a.total_q = static_cast<int32_t>(total_q);
  a.total_k = static_cast<int32_t>(total_k);
  a.hk = d.k_heads;
  a.group = group;
  a.tok = tok;
  a.causal = d.causal;
  a.div_hk = lgt::magic_encode(static_cast<uint32_t>(d.k_heads));
  a.div_group = lgt::magic_encode(static_cast<uint32_t>(group));
  a.div_pair = lgt::magic_encode(static_cast<uint32_t>(2 * tok));
  a.cs = (d.scale > 0.0f ? d.scale : 1.0f / std::sqrt(static_cast<float>(d.head_dim))) * 1.4426950408889634f;
  const bool bf16 = d.dtype == GEMM_BF16;
  a.idesc_s = lgt::idesc_f16(bf16, 0u, 0u, lgt::kPrRows, lgt::kPrKeys);
  a.idesc_pv = lgt::idesc_f16(bf16, 0u, 1u, lgt::kPrRows, static_cast<uint32_t>(d.head_dim));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(units);
  const cudaError_t e = d.head_dim == 128
                            ? (bf16 ? lgt::launch_prompt<128, true>(a, grid, s) : lgt::launch_prompt<128, false>(a, grid, s))
                            : (bf16 ? lgt::launch_prompt<64, true>(a, grid, s) : lgt::launch_prompt<64, false>(a, grid, s));
  if (e != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  return GEMM_OK;
}

gemm_status_t attn_prompt_sync_status(attn_prompt_plan_t* plan, void* stream) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return GEMM_ERR_CUDA;
  lgt::DeviceStatus st;
  if (cudaMemcpy(&st, plan->d_status, sizeof(st), cudaMemcpyDeviceToHost) != cudaSuccess) return GEMM_ERR_CUDA;
  if (st.code != 0) {
    if (cudaMemset(plan->d_status, 0, sizeof(st)) != cudaSuccess) return GEMM_ERR_CUDA;
    return static_cast<gemm_status_t>(st.code);
  }
  return GEMM_OK;
}

gemm_status_t attn_prompt_destroy(attn_prompt_plan_t* plan) {
  if (!plan) return GEMM_OK;
  if (plan->d_status) cudaFree(plan->d_status);
  delete plan;
  return GEMM_OK;
}

}  // extern "C"
