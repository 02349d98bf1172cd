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
//                  it by 2^8; P goes back to tensor memory in 16 bits, each
//                  half as soon as it is made.
//   O += P V       tcgen05, A = P from tensor memory, B = V as it lies
//                  (MN-major).
// The two tiles alternate: while the tensor core works on one tile's
// products, the other tile's softmax runs.
//
// Few rows.  Where a unit's tokens fit one tile, both tiles take them, each
// every other block of the keys, and the two results are joined at the end:
// the walk over the keys, which is what such a unit takes, is half as long.
// Where there are few units, a sequence whose walk over its keys is longer than
// twice what each SM would have to do is cut into units of T tokens, so that
// all of them are of this kind.  (A kernel of its own, kPrFew: in the other the
// code that no unit uses costs 2 %.)  Where there are so few that most SMs would
// have none, the keys of a unit are cut over a cluster of two to eight CTAs
// (kPrCut); each leaves its sums in its shared memory, and the cluster joins
// them, a share of the columns a CTA, in the order of the keys.
//
// Work.  A unit is 2T tokens (or T) of a sequence and a key head.  The grid has a
// block for every unit, the ones with the most keys of a sequence first; a
// running CTA takes over blocks that have not started (cluster launch
// control) shortly before it is done with its own, so that it loads the next
// unit's tiles and issues their first products while the softmax warps still
// write the last unit's result.
//
// Warps (384 threads): 0-3 softmax of tile 0, 4-7 of tile 1, 8 loads K,
// 9 issues the products, 11 finds the units and loads Q, 10 loads V (three
// warps load because issuing a copy holds its thread for 250 cycles or more)
// and looks over the rows of it that some query of the CTA must not see, since
// a weight of 0 does not cancel an infinity or a NaN: rows that no query sees
// (later ones, or the next sequence's) are cleared; in the others (2T at most)
// values that are not finite are, and are added to the results of the queries
// that do see them at the end, where a sum with a positive weight would have
// left the same.
// Tensor memory: S of the tiles at columns 0 and 128, O at 256 and
// 256 + head_dim; P lies over its own S (head_dim 128: the columns are all
// taken; the products that read P and write the next S are of one shape and
// one issuing thread, which keeps them in order) or behind O (head_dim 64).
// Every wait is bounded; one that runs out records GEMM_ERR_TIMEOUT and the
// CTA winds down.
//
// Bound: the tensor core, whose S reads all of the shared memory's rate (8 KiB
// in 64 cycles), and in long runs the power limit.  Measured (bf16, head_dim
// 128, causal, visible products only): 4 prompts of 4096, 32 / 8 heads, 334 us,
// 1646 TFLOP/s, 86 % of cuBLAS's burst rate (372 us in long runs); 1 of 16384,
// 16 / 2 heads, 620 us, 1773 TFLOP/s, 92 % (tensor pipe 83 % of cycles).  Steps
// of the latter: products issued by a whole warp, maximum before weights 718;
// maximum beside weights, halves handed over 680; one issuing thread, waits
// ahead 646; constant ring places 619.  Short ones are bound by the walk of a
// CTA over its keys: 1.25 us a block of 128 for both tiles (1 at head_dim 64),
// 6 us at the ends.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <cstdlib>
#include <new>
#include <type_traits>

#include "attn_prompt.h"
#include "half_types.cuh"
#include "kernels.h"
#include "plan.h"
#include "ptx.cuh"

namespace lgt {
namespace {

constexpr int kPrThreads = 384;  // 168 registers each
constexpr int kPrRows = 128;     // rows of a tile
constexpr int kPrKeys = 128;     // keys of a block
constexpr int kPrTimeout = GEMM_ERR_TIMEOUT;
constexpr float kPrLazy = 8.0f;
// Blocks of keys before a unit's end at which the next one is taken: soon
// enough that its tiles are there when the tensor core is free, and not while
// another CTA would come to it earlier.  (us, taken at once and so: one prompt of
// 2048 tokens, 32 / 8 heads of 128, 39.1 and 31.4; 13 ragged ones, 12 / 4 of 64,
// 23.1 and 20.2; 4 of 4096 338 and 334.  Between one and six blocks it is the
// same but for the ragged ones: 20.8 to 19.6.)
constexpr int kPrClaim = 4;
// Units an SM below which the kernel for few is taken.  (us with one, two and
// four: 13 ragged prompts 24.0, 16.7, 16.7; 13 of up to 766 after about 1400, 28 /
// 4 heads of 64, 50.3, 50.3, 46.7; one of 3431, 32 / 4, 58.5, 58.5, 61.7; one of
// 4096, 32 / 8 heads of 128, 53.9, 53.9, 56.4.)
constexpr int kPrFill = 2;
constexpr int kPrParts = 8;    // CTAs of a cluster that may share a unit
// Blocks of keys, in the mean, that sharing takes from a CTA's walk at least:
// the cluster's start and join cost 1.5 us with a row, 2.5 with all, what two
// pairs of blocks do.  (us, shared and not: 1 token after about 4096 keys, 32 /
// 8 heads of 128, 8.7 and 18.4, after 32768 23.6 and 120; 64 after 8192 17.2 and
// 33.7; 512 after about 400, 8 / 2 heads, 11.0 and 11.1; 1000 after none, 8 / 8
// heads, where sharing spares 4, 14.3 and 12.8.)
constexpr int kPrSpare = 5;

// The kernels: for many units, for few (of one tile where walks are long),
// and for so few that the keys of each are cut over a cluster.
enum PromptKind { kPrMany, kPrFew, kPrCut };

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
  int32_t sms;
  int32_t causal;
  int32_t lg_parts;  // log2 of the CTAs that share a unit
  int32_t withhold;  // test aid: CTA 0 never makes its first load of K
  MagicDiv div_hk, div_group, div_tok, div_pair;  // by T, by 2T
  float cs;  // scale * log2(e)
  uint32_t idesc_s, idesc_pv;
};

// Sequences of a call: a CTA's way through the cumulative lengths, 0.7 us for 32
// of them, is far within the limit of its waits.
constexpr int kPrMaxBatch = 1 << 20;

// What a CTA works on, 2T tokens of one sequence and key head, and what
// follows from that for its tiles and blocks of keys.
struct PromptUnit {
  int row0, tokens;        // first row of Q, tokens (1 .. 2T); 0: nothing, -1: no more units
  int key_row, nk;         // first row of K and V, keys
  int shift;               // token i of the unit sees keys <= i + shift
  int h;                   // key head
  // tokens of the tiles, and blocks with keys that they see; with split = 1
  // the tokens are both tiles' and the blocks are dealt in turns, the first
  // one to tile `start`
  int toks[2], blocks[2];
  int nb, split, start;    // nb: blocks of the unit
  // keys that every token sees, and that any does; the blocks from `mixed` on
  // (three at most: they span 2T keys) hold some that not all see
  int all_see, any_sees, mixed;
  int odd;                 // V held values that are not finite
  int from, keys;          // first key of the part that this CTA has (key_row, nk and shift are the part's), and all keys
  int pad[13];
};
static_assert(sizeof(PromptUnit) == 128, "two of them in shared memory");

template <PromptKind KIND>
__device__ __forceinline__ void shape_unit(const PromptArgs& a, PromptUnit& x, int turn) {
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    x.toks[t] = min(max(x.tokens - t * a.tok, 0), a.tok);
    const int last = t * a.tok + x.toks[t] - 1;
    const int vis = x.toks[t] == 0 ? 0 : a.causal ? min(max(last + x.shift + 1, 0), x.nk) : x.nk;
    x.blocks[t] = (vis + kPrKeys - 1) / kPrKeys;
  }
  x.nb = max(x.blocks[0], x.blocks[1]);
  x.split = KIND != kPrMany && x.tokens <= a.tok;
  x.start = turn;
  if (x.split) {
    x.toks[1] = x.toks[0];
    x.blocks[0] = (x.nb + (turn ^ 1)) / 2;
    x.blocks[1] = (x.nb + turn) / 2;
  }
  x.all_see = a.causal ? min(max(x.shift + 1, 0), x.nk) : x.nk;
  x.any_sees = a.causal ? min(max(x.tokens + x.shift, 0), x.nk) : x.nk;
  x.mixed = x.all_see / kPrKeys;
}

// Part `rank` of the unit's blocks of keys, as a unit of its own.
__device__ __forceinline__ void cut_unit(const PromptArgs& a, PromptUnit& x, int rank) {
  const int sees = a.causal ? min(max(x.tokens + x.shift, 0), x.nk) : x.nk;
  const int nb = (sees + kPrKeys - 1) / kPrKeys;
  const int b0 = (nb * rank) >> a.lg_parts, b1 = (nb * (rank + 1)) >> a.lg_parts;
  x.keys = x.nk;
  x.from = b0 * kPrKeys;
  x.nk = min(x.nk, b1 * kPrKeys) - min(x.nk, x.from);
  x.key_row += x.from;
  x.shift -= x.from;
}

template <int D, PromptKind KIND>
struct PromptCfg {
  static constexpr uint32_t CHUNK = 128u * 128u;      // 64 values of 128 rows
  static constexpr uint32_t TILE = (D / 64) * CHUNK;  // a tile of Q, K or V
  // Blocks of K and of V in the ring.  Where a unit's two tiles take every other
  // block, a place is free for the time of one product only: four of each and
  // a small loop that issues the products (its instructions are fetched again
  // each time round) against two and one stretch of code a place, head_dim 64:
  // 13 ragged prompts 15.4 us and 16.8, single queries 16.5 and 18.0.  The
  // kernel for many units: 153 us so and 97.7 (8 x 512 tokens after 1500 to 3000).
  static constexpr uint32_t TURNS = D == 64 && KIND != kPrMany ? 4 : 2;
  static constexpr bool UNROLL = TURNS == 2;
  static constexpr int NS = 2 * static_cast<int>(TURNS);                // its places: K, V, K, V, ...
  static constexpr uint32_t Q_OFF = 0;                // two tiles
  static constexpr uint32_t RING_OFF = 2 * TILE;
  static constexpr uint32_t BAR_OFF = RING_OFF + NS * TILE;
  // full[NS], empty[NS], q_full[2], q_empty[2], s_full[2], p_full[2][2], o_full[2], v_clean[2][3],
  // unit_full[2], unit_empty[2], taken, teardown, join_ready[2][4], join_done[2][4], near_end
  static constexpr int NBARS = 2 * NS + 41;
  static constexpr uint32_t TAKEN_OFF = BAR_OFF + ((NBARS * 8 + 15) & ~15);  // 16 bytes: a block taken over
  static constexpr uint32_t UNIT_OFF = TAKEN_OFF + 16;                       // two PromptUnit
  static constexpr uint32_t XCH_OFF = UNIT_OFF + 2 * sizeof(PromptUnit);     // {m, l} of both tiles' rows
  static constexpr uint32_t MISC_OFF = XCH_OFF + 2 * kPrRows * 8;
  static constexpr uint32_t SMEM = MISC_OFF + 16 + 1024;  // slack for the 1024-byte alignment
  // A part's sums, where the ring was: four columns of all rows, the next four
  // (apart by a place more than the rows, for the banks), ..., {m, l} of the rows.
  static constexpr uint32_t PART_OFF = RING_OFF, PART_STEP = (kPrRows + 1) * 16u;
  static constexpr uint32_t PART_ML_OFF = PART_OFF + (D / 4) * PART_STEP;
  static_assert(PART_ML_OFF + kPrRows * 8 <= RING_OFF + NS * TILE, "a part's sums");
  static constexpr uint32_t S_COL = 128;                  // between the tiles' S
  static constexpr uint32_t O_COL = 256;
  static constexpr uint32_t P_COL = D == 128 ? 0 : 384;
  static constexpr uint32_t P_STEP = D == 128 ? 128 : 64;
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

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

__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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

// The bounded wait, all but its first try out of line: it stands at many
// places, in code that several warps run through at once.
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, uint64_t limit_ns, volatile int* abort_flag) {
  return mbar_wait_bounded(bar, parity, limit_ns, abort_flag);
}
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, uint64_t limit_ns, volatile int* abort_flag) {
  return mbar_try_wait(bar, parity) || wait_on(bar, parity, limit_ns, abort_flag);
}

// A bounded wait whose outcome is the whole warp's: a lane that gave up while
// another saw the phase complete would part from it at the next warp barrier.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, wait_bounded(bar, parity, limit_ns, abort_flag));
}

// Ask for a block of the grid that has not started; the answer's 16 bytes
// arrive at `dst` and complete on `bar`.
__device__ __forceinline__ void take_block(uint32_t dst, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(dst),
               "r"(bar)
               : "memory");
}
// Its index, or -1 where there is none.
__device__ __forceinline__ int64_t taken_block(uint32_t src) {
  uint32_t ok, x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(ok), "=r"(x)
      : "r"(src)
      : "memory");
  return ok ? static_cast<int64_t>(x) : -1;
}

// Query and key rows of sequence b.
struct PromptSeq {
  int q0, nq, k0, nk;
};
__device__ __forceinline__ PromptSeq seq_at(const PromptArgs& a, int b) {
  PromptSeq s{0, 0, 0, 0};
  if (b < a.batch) {
    s.q0 = min(max(a.cu_q[b], 0), a.total_q);
    s.nq = max(min(a.cu_q[b + 1], a.total_q) - s.q0, 0);
    s.k0 = min(max(a.cu_k[b], 0), a.total_k);
    s.nk = max(min(a.cu_k[b + 1], a.total_k) - s.k0, 0);
  }
  return s;
}

// Blocks of keys above which a sequence is cut into units of one tile: twice
// the blocks that each SM would walk if all units were of two.  (Measured,
// 32 / 8 heads of 128: one prompt of 512 tokens 10.7 us so cut, 12.0 not; one
// of 64 after 8192 keys 35 and 58; four of 256, which it leaves alone, 13.0
// and 9.8.)  The whole warp returns the same.
// (mine: this lane's of the first 32 sequences, here and below.)
__device__ __forceinline__ int narrow_above(const PromptArgs& a, const PromptSeq& mine) {
  float sum = 0.0f;
  for (int b = threadIdx.x & 31; b < a.batch; b += 32) {
    const PromptSeq s = b < 32 ? mine : seq_at(a, b);
    const float walk = static_cast<float>(s.nk) - (a.causal ? 0.5f * static_cast<float>(s.nq) : 0.0f);
    sum += static_cast<float>(magic_div(static_cast<uint32_t>(s.nq + 2 * a.tok) - 1u, a.div_pair)) *
           (fmaxf(walk, 0.0f) * (1.0f / kPrKeys) + 0.5f);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return static_cast<int>(fminf(2.0f * sum * static_cast<float>(a.hk) / static_cast<float>(a.sms), 1e9f));
}

// Where in the list of units a warp is: 32 sequences from b0 on, this lane's of
// them, and the units before them.  Blocks are taken over in their order, so the
// search for the next unit goes on from here, and a CTA goes through the batch
// once.  (From the first sequence on for each unit it is the batch squared:
// 4096 sequences of one token, 4 / 1 heads of 64, 421 us and 97, 16384 5700 and 357.)
struct PromptPlace {
  int b0;
  uint32_t before;
  PromptSeq seq;
};

// Unit `u` of the list (sequences in order, each one's last tokens -- the
// most keys -- first); every lane of the warp returns the same.
__device__ __forceinline__ PromptUnit find_unit(const PromptArgs& a, uint32_t u, int narrow, PromptPlace& at) {
  const int lane = threadIdx.x & 31;
  PromptUnit r{};
  bool moved = u < at.before;  // (no order of the takeovers is promised)
  if (moved) at.b0 = 0, at.before = 0u;
  for (; at.b0 < a.batch; at.b0 += 32) {
    if (moved) at.seq = seq_at(a, at.b0 + lane);
    moved = true;
    const PromptSeq& q = at.seq;
    const bool cut = (q.nk + kPrKeys - 1) / kPrKeys > narrow;
    const int my_span = cut ? a.tok : 2 * a.tok;
    const uint32_t n = magic_div(static_cast<uint32_t>(q.nq + my_span) - 1u, cut ? a.div_tok : a.div_pair);
    uint32_t x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const uint32_t all = __shfl_sync(0xffffffffu, x, 31);
    if (u - at.before < all) {  // (u >= before)
      const uint32_t in = u - at.before;
      const unsigned hit = __ballot_sync(0xffffffffu, x > in);
      const int src = __ffs(hit) - 1;
      auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, src); };
      const uint32_t units = __shfl_sync(0xffffffffu, n, src), first = __shfl_sync(0xffffffffu, x - n, src);
      const int span = of(my_span), nq = of(q.nq);
      const int i0 = static_cast<int>(units - 1u - (in - first)) * span;
      r.row0 = of(q.q0) + i0;
      r.tokens = min(span, nq - i0);
      r.key_row = of(q.k0);
      r.nk = of(q.nk);
      r.shift = i0 + r.nk - nq;
      return r;
    }
    at.before += all;
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

// Add the values of V that are not finite to a row's sums: two columns', 32
// columns' (at `p`).  (They stay what they are, or become NaN, in the division
// by the row's sum of weights.)
template <bool BF16>
__device__ __forceinline__ void add_odd_pair(uint32_t x, float& s0, float& s1) {
  const uint32_t bad = odd_halves<BF16>(x);
  const float2 y = unpack_pair16<BF16>(x);
  if (bad & 0x8000u) s0 += y.x;
  if (bad & 0x80000000u) s1 += y.y;
}
template <bool BF16>
__device__ __forceinline__ void add_odd(const uint16_t* p, uint32_t (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float s0 = __uint_as_float(v[2 * i]), s1 = __uint_as_float(v[2 * i + 1]);
    add_odd_pair<BF16>(reinterpret_cast<const uint32_t*>(p)[i], s0, s1);
    v[2 * i] = __float_as_uint(s0);
    v[2 * i + 1] = __float_as_uint(s1);
  }
}

// Four lanes' 16-byte pieces (four of four words each) transposed: lane q
// gets piece q of its neighbours' rows 0 .. 3.
__device__ __forceinline__ void exchange4(uint32_t (&y)[16], int lane) {
  const bool up2 = lane & 2, up1 = lane & 1;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, up2 ? y[i] : y[i + 8], 2);
    if (up2) y[i] = got; else y[i + 8] = got;
  }
#pragma unroll
  for (int i = 0; i < 16; i += 8)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, up1 ? y[i + e] : y[i + 4 + e], 1);
      if (up1) y[i + e] = got; else y[i + 4 + e] = got;
    }
}

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster_v2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Join the 2^LG parts of a unit: this CTA, `rank` of the cluster, has its share
// of the columns.  A thread takes four columns of kU rows at a time, so that
// kPrParts loads are on their way whatever the parts are, and adds the parts in
// the order of the keys.
template <int D, bool BF16, int LG>
__device__ __forceinline__ void join_parts(const PromptArgs& a, const PromptUnit& w, uint32_t base, uint32_t rank) {
  using C = PromptCfg<D, kPrCut>;
  constexpr int P = 1 << LG, kU = kPrParts / P, kShare = D / 4 / P;
  const int items = w.toks[0] * a.group * kShare;
  uint32_t odd = 0;
#pragma unroll
  for (int p = 0; p < P; ++p)
    odd |= ld_cluster_u32(mapa_shared(base + C::UNIT_OFF + static_cast<uint32_t>(offsetof(PromptUnit, odd)), p));
  for (int i0 = threadIdx.x; i0 < items; i0 += kPrThreads * kU) {
    float2 ml[kU][P];
    float4 x[kU][P];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int i = min(i0 + u * kPrThreads, items - 1), row = i / kShare, c4 = static_cast<int>(rank) * kShare + i % kShare;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        ml[u][p] = ld_cluster_v2(mapa_shared(base + C::PART_ML_OFF + row * 8, p));
        x[u][p] = ld_cluster_v4(mapa_shared(base + C::PART_OFF + c4 * C::PART_STEP + row * 16, p));
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int i = i0 + u * kPrThreads, row = i / kShare, c4 = static_cast<int>(rank) * kShare + i % kShare;
      if (i >= items) break;
      float top = -INFINITY, l = 0.0f;
#pragma unroll
      for (int p = 0; p < P; ++p) top = fmaxf(top, ml[u][p].x);
      const float ref = top == -INFINITY ? 0.0f : top;
      float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const float f = ex2(ml[u][p].x - ref);
        l = fmaf(ml[u][p].y, f, l);
        sum = make_float4(fmaf(x[u][p].x, f, sum.x), fmaf(x[u][p].y, f, sum.y), fmaf(x[u][p].z, f, sum.z),
                          fmaf(x[u][p].w, f, sum.w));
      }
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      sum = make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
      uint32_t tok, g;
      magic_divmod(static_cast<uint32_t>(row), a.div_group, tok, g);
      if (odd) {
        const int shift = w.shift + w.from;
        const int vis = a.causal ? min(static_cast<int>(tok) + shift + 1, w.keys) : w.keys;
        for (int k = a.causal ? min(max(shift + 1, 0), w.keys) : w.keys; k < vis; ++k) {
          const uint32_t* v = reinterpret_cast<const uint32_t*>(a.v + static_cast<int64_t>(w.key_row - w.from + k) * a.vs +
                                                                w.h * D + c4 * 4);
          add_odd_pair<BF16>(v[0], sum.x, sum.y);
          add_odd_pair<BF16>(v[1], sum.z, sum.w);
        }
      }
      const uint2 y = l == 0.0f ? make_uint2(0u, 0u)
                                : make_uint2(pack_pair16<BF16>(sum.x, sum.y), pack_pair16<BF16>(sum.z, sum.w));
      *reinterpret_cast<uint2*>(a.out + static_cast<int64_t>(w.row0 + static_cast<int>(tok)) * a.os +
                                static_cast<int64_t>(w.h * a.group + static_cast<int>(g)) * D + c4 * 4) = y;
    }
  }
}

template <int D, bool BF16, PromptKind KIND>
__global__ void __launch_bounds__(kPrThreads, 1) prompt_kernel(const __grid_constant__ PromptArgs a) {
  using C = PromptCfg<D, KIND>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw_base);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

  const uint32_t bar0 = base + C::BAR_OFF;
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (C::NS + s); };
  constexpr int kB = 2 * C::NS;
  auto q_full = [&](int t) { return bar0 + 8u * (kB + t); };
  auto q_empty = [&](int t) { return bar0 + 8u * (kB + 2 + t); };
  auto s_full = [&](int t) { return bar0 + 8u * (kB + 4 + t); };
  auto p_full = [&](int t, int half) { return bar0 + 8u * (kB + 6 + 2 * t + half); };
  auto o_full = [&](int t) { return bar0 + 8u * (kB + 10 + t); };
  // (of even and odd units: a unit is taken up only when nobody is at the one
  // before the last, so no wait can be two phases behind)
  auto v_clean = [&](int i) { return bar0 + 8u * (kB + 12 + i); };
  auto unit_full = [&](int i) { return bar0 + 8u * (kB + 18 + i); };
  auto unit_empty = [&](int i) { return bar0 + 8u * (kB + 20 + i); };
  const uint32_t taken = bar0 + 8u * (kB + 22);
  const uint32_t teardown = bar0 + 8u * (kB + 23);
  auto join_ready = [&](int t, int q) { return bar0 + 8u * (kB + 24 + t * 4 + q); };
  auto join_done = [&](int t, int q) { return bar0 + 8u * (kB + 32 + t * 4 + q); };
  const uint32_t near_end = bar0 + 8u * (kB + 40);
  PromptUnit* units = reinterpret_cast<PromptUnit*>(smem + C::UNIT_OFF);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(q_full(t), 1);
      mbar_init(q_empty(t), 1);
      mbar_init(s_full(t), 1);
      mbar_init(p_full(t, 0), 4);  // the tile's softmax warps
      mbar_init(p_full(t, 1), 4);
      mbar_init(o_full(t), 1);
      mbar_init(unit_full(t), 1);
      mbar_init(unit_empty(t), 11);  // eight softmax warps, loads, products, V
    }
    for (int i = 0; i < 6; ++i) mbar_init(v_clean(i), 1);
    for (int i = 0; i < 8; ++i) {
      mbar_init(join_ready(i >> 2, i & 3), 1);
      mbar_init(join_done(i >> 2, i & 3), 1);
    }
    mbar_init(taken, 1);
    mbar_init(near_end, 1);
    mbar_init(teardown, 1);
    *abort_flag = 0;
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

  // Where P does not lie over S, a tile's next S is issued as soon as the first
  // half of P says that S has been read, and o_full is of every block.  (8 x 512
  // tokens after 1500 to 3000, 32 / 8 heads of 64: 97.7 us, after the product 102.8.)
  constexpr bool kApart = C::P_COL != 0;

  // Every role walks the same list of units; it and every ring and barrier go
  // on from one unit to the next, so each role counts its own uses of them.
  const uint64_t limit = a.wait_limit_ns;
  auto unit_ready = [&](int it) { return warp_wait(unit_full(it & 1), (it >> 1) & 1, limit, abort_flag); };
  uint32_t issued = 0;                 // loads of K (warp 8), of V (warp 10)
  int q_uses[2] = {0, 0};         // loads of Q (warp 11)
  int asked = 0;                  // blocks asked for (warp 11)

  auto withheld = [&](int which, uint32_t n) { return a.withhold && blockIdx.x == 0 && which == 0 && n == 0; };
  // Load block j of K (which = 0) or V (1) of unit w into its next place.
  auto load = [&](int which, int j, const PromptUnit& w, const CUtensorMap* map, bool leader) {
    const uint32_t s = 2 * (issued % C::TURNS) + which;
    if (issued >= C::TURNS && !warp_wait(empty(s), (issued / C::TURNS - 1) & 1, limit, abort_flag)) return false;
    if (leader && !withheld(which, issued)) {
      mbar_arrive_expect_tx(full(s), C::TILE);
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        tma_load_3d(base + C::RING_OFF + s * C::TILE + c * C::CHUNK, map, full(s), c * 64, w.h, w.key_row + j * kPrKeys);
    }
    __syncwarp();
    ++issued;
    return true;
  };

  if (warp == 8) {
    // -------------------------------------------------------- loads of K
    const bool leader = elect_one();
    bool ok = true;
    for (int it = 0; ok; ++it) {
      if (!(ok = unit_ready(it))) break;
      const PromptUnit w = units[it & 1];
      if (w.tokens < 0) break;
      for (int j = 0; ok && j < w.nb; ++j) {
        if (!(ok = load(0, j, w, &a.tm_k, leader))) break;
        if (j == max(w.nb - kPrClaim, 0) && lane == 0) mbar_arrive(near_end);
      }
      if (w.nb == 0 && lane == 0) mbar_arrive(near_end);
      if (lane == 0) mbar_arrive(unit_empty(it & 1));
    }
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
        if (ok) ok = wait_bounded(bar, parity, limit, abort_flag);
        return ok;
      };
      // (this thread is the pace of the CTA: blocks are taken by turns with the
      // ring's places for K and for V, and where there are two of each, every
      // address is a constant in the code of its turn)
      auto wait_full = [&](int slot, uint32_t block) { return wait(full(slot), block / C::TURNS & 1u); };
      // 16 values of d are 32 bytes further in a 64-value chunk
      const uint64_t q_desc = sw128_desc(base + C::Q_OFF, 16u, 1024u), k_desc = sw128_desc(base + C::RING_OFF, 16u, 1024u);
      const uint64_t v_desc = sw128_desc(base + C::RING_OFF, C::CHUNK, 1024u);
      const uint32_t idesc_s = a.idesc_s, idesc_pv = a.idesc_pv;
      auto issue_s = [&](int t, int q_tile, int slot) {
        const uint64_t qd = q_desc + q_tile * (C::TILE >> 4), kd = k_desc + slot * (C::TILE >> 4);
        const uint32_t dst = tmem + t * C::S_COL;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t off = ((k >> 2) * C::CHUNK + (k & 3) * 32u) >> 4;
          tc_mma_f16_ss(dst, qd + off, kd + off, idesc_s, k > 0 ? 1u : 0u);
        }
        tc_commit(s_full(t));
      };
      auto issue_pv = [&](int t, int slot, int half, bool first) {
        const uint64_t vd = v_desc + slot * (C::TILE >> 4);
        const uint32_t dst = tmem + C::O_COL + t * D, pa = tmem + C::P_COL + t * C::P_STEP;
        // 16 keys are 2 KiB of V and 8 columns of P
#pragma unroll
        for (int i = 0; i < kPrKeys / 32; ++i) {
          const uint32_t k = half * (kPrKeys / 32) + i;
          mma_ts(dst, pa + k * 8, vd + static_cast<uint64_t>(k * 2048u >> 4), idesc_pv, (first && i == 0) ? 0u : 1u);
        }
      };
      uint32_t p_parity = 0, q_parity = 0;  // a bit a tile
      uint32_t v_parity = 0;      // of the uses of v_clean
      uint32_t block = 0;         // of the CTA's, counted through
      int nb = 0, mixed = 0, blocks[2] = {0, 0}, it = 0;
      auto first_s = [&](auto turn) {
        const int ks = 2 * turn;
        if (!wait_full(ks, block)) return;
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (blocks[t] > 0 && wait(q_full(t), q_parity >> t & 1u)) {
            q_parity ^= 1u << t;
            tc_fence_after();
            issue_s(t, t, ks);
            if (blocks[t] == 1) tc_commit(q_empty(t));
          }
        if (ok) tc_commit(empty(ks));
        wait_full(ks + 1, block);
      };
      auto step = [&](auto turn, int j) {
        const int vs = 2 * turn + 1, ks = 2 * ((turn + 1) % static_cast<int>(C::TURNS));
        const bool more = j + 1 < nb;
        if (j >= mixed) {
          const int i = (it & 1) * 3 + j - mixed;
          if (!wait(v_clean(i), (v_parity >> i) & 1u)) return;
          v_parity ^= 1u << i;
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          auto next_s = [&] {
            if (j + 1 >= blocks[t]) return;
            issue_s(t, t, ks);
            if (j + 2 == blocks[t]) tc_commit(q_empty(t));
          };
          if (j < blocks[t]) {
            if (!wait(p_full(t, 0), p_parity >> t & 1u)) return;
            tc_fence_after();
            issue_pv(t, vs, 0, j == 0);
            if (t == 0 && more && !wait_full(ks, block + 1)) return;
            if (kApart) next_s();
            if (!wait(p_full(t, 1), p_parity >> t & 1u)) return;
            tc_fence_after();
            issue_pv(t, vs, 1, false);
            p_parity ^= 1u << t;
            if (kApart || j + 1 == blocks[t]) tc_commit(o_full(t));
          } else if (t == 0 && more && !wait_full(ks, block + 1)) {
            return;
          }
          if (t == 1) tc_commit(empty(vs));
          if (t == 1 && more && !wait_full(ks + 1, block + 1)) return;
          if (!kApart) next_s();
        }
        if (more) tc_commit(empty(ks));
      };
      // The same for units whose tiles share their rows: blocks go to the tile
      // of their place in the ring, so the tile is the turn.
      auto first_s_split = [&](auto turn, int j) {
        const int t = turn % 2, ks = 2 * turn;
        if (!wait_full(ks, block + j)) return;
        tc_fence_after();
        issue_s(t, 0, ks);
        tc_commit(empty(ks));
        if (j + 1 == nb) tc_commit(q_empty(0));
      };
      auto step_split = [&](auto turn, int j) {
        const int t = turn % 2, vs = 2 * turn + 1, ks = 2 * ((turn + 2) % static_cast<int>(C::TURNS));
        if (!wait_full(vs, block)) return;
        if (j >= mixed) {
          const int i = (it & 1) * 3 + j - mixed;
          if (!wait(v_clean(i), (v_parity >> i) & 1u)) return;
          v_parity ^= 1u << i;
        }
        if (!wait(p_full(t, 0), p_parity >> t & 1u)) return;
        tc_fence_after();
        issue_pv(t, vs, 0, j < 2);
        if (j + 2 < nb && !wait_full(ks, block + 2)) return;
        auto next_s = [&] {
          if (j + 2 >= nb) return;
          issue_s(t, 0, ks);
          tc_commit(empty(ks));
          if (j + 3 == nb) tc_commit(q_empty(0));
        };
        if (kApart) next_s();
        if (!wait(p_full(t, 1), p_parity >> t & 1u)) return;
        tc_fence_after();
        issue_pv(t, vs, 1, false);
        p_parity ^= 1u << t;
        if (kApart || j + 2 >= nb) tc_commit(o_full(t));
        tc_commit(empty(vs));
        if (!kApart) next_s();
      };
      // (written out: one more lambda around them costs the kernel for many 5 %
      // at head_dim 64)
      constexpr std::integral_constant<int, 0> even{};
      constexpr std::integral_constant<int, 1> odd{};
      auto turn_of = [](uint32_t n) { return static_cast<int>(n % C::TURNS); };
      for (; ok; ++it) {
        if (!wait(unit_full(it & 1), (it >> 1) & 1)) break;
        nb = units[it & 1].nb;
        mixed = units[it & 1].mixed;
        blocks[0] = units[it & 1].blocks[0];
        blocks[1] = units[it & 1].blocks[1];
        if (units[it & 1].tokens < 0) break;
        if (KIND != kPrMany && units[it & 1].split) {
          if (nb > 0 && wait(q_full(0), q_parity & 1u)) {
            q_parity ^= 1u;
            for (int j = 0; ok && j < min(nb, 2); ++j) {
              if constexpr (!C::UNROLL)
                first_s_split(turn_of(block + j), j);
              else if ((block + j) & 1u)
                first_s_split(odd, j);
              else
                first_s_split(even, j);
            }
          }
          for (int j = 0; ok && j < nb; ++j, ++block) {
            if constexpr (!C::UNROLL)
              step_split(turn_of(block), j);
            else if (block & 1u)
              step_split(odd, j);
            else
              step_split(even, j);
          }
        } else {
          if (nb > 0) {
            if constexpr (!C::UNROLL)
              first_s(turn_of(block));
            else if (block & 1u)
              first_s(odd);
            else
              first_s(even);
          }
          for (int j = 0; ok && j < nb; ++j, ++block) {
            if constexpr (!C::UNROLL)
              step(turn_of(block), j);
            else if (block & 1u)
              step(odd, j);
            else
              step(even, j);
          }
        }
        mbar_arrive(unit_empty(it & 1));
      }
      if (!ok && !*abort_flag) prompt_timeout(a, abort_flag, 1);
      tc_commit(teardown);  // every product is done before the tensor memory is freed
    }
    __syncwarp();
  } else if (warp == 10) {
    // ------------------- loads of V, and its rows that not all queries see
    const bool leader = elect_one();
    bool ok = true;
    for (int it = 0; ok; ++it) {
      if (!(ok = unit_ready(it))) break;
      PromptUnit* unit = &units[it & 1];
      const PromptUnit w = *unit;
      if (w.tokens < 0) break;
      // (block j is looked over after j + 1 is asked for)
      for (int j = 0; ok && j <= w.nb; ++j) {
        if (j < w.nb && !(ok = load(1, j, w, &a.tm_v, leader))) break;
        const int jj = j - 1;
        if (jj < w.mixed || jj < 0) continue;
        const uint32_t n = issued - (j < w.nb ? 2u : 1u), s = 2 * (n % C::TURNS) + 1;
        if (!(ok = warp_wait(full(s), n / C::TURNS & 1, limit, abort_flag))) break;
        const uint32_t vb = base + C::RING_OFF + s * C::TILE;
        const int look = max(w.all_see - jj * kPrKeys, 0), clear = min(w.any_sees - jj * kPrKeys, kPrKeys);
        uint32_t odd = 0;
        for (int r = look * 8 + lane; r < clear * 8; r += 32) {
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const uint32_t at = vb + c * C::CHUNK + r * 16;
            const uint4 v = ld_shared_v4(at);
            const uint32_t o0 = odd_halves<BF16>(v.x), o1 = odd_halves<BF16>(v.y), o2 = odd_halves<BF16>(v.z),
                           o3 = odd_halves<BF16>(v.w);
            if (o0 | o1 | o2 | o3) {
              odd = 1;
              st_shared_v4(at, v.x & ~spread_halves(o0), v.y & ~spread_halves(o1), v.z & ~spread_halves(o2),
                           v.w & ~spread_halves(o3));
            }
          }
        }
        for (int r = clear * 8 + lane; r < kPrKeys * 8; r += 32)
#pragma unroll
          for (int c = 0; c < D / 64; ++c) st_shared_v4(vb + c * C::CHUNK + r * 16, 0u, 0u, 0u, 0u);
        if (odd) *const_cast<volatile int*>(&unit->odd) = 1;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_clean((it & 1) * 3 + jj - w.mixed));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(unit_empty(it & 1));
    }
    if (!ok && lane == 0 && !*abort_flag) prompt_timeout(a, abort_flag, 3);
  } else if (warp == 11) {
    // ------------------------------------------------- units, loads of Q
    int64_t block = KIND == kPrCut ? blockIdx.x >> a.lg_parts : blockIdx.x;
    int turn = 0;  // of the next unit's first block at the ring's places
    PromptPlace place{0, 0u, seq_at(a, lane)};
    const int narrow = KIND == kPrFew ? narrow_above(a, place.seq) : KIND == kPrCut ? -1 : 0x7fffffff;
    bool ok = true;
    int it = 0;
    auto publish = [&](const PromptUnit& w) {
      if (it >= 2 && !(ok = warp_wait(unit_empty(it & 1), ((it >> 1) - 1) & 1, limit, abort_flag))) return;
      if (lane == 0) {
        units[it & 1] = w;
        mbar_arrive(unit_full(it & 1));
      }
      __syncwarp();
      ++it;
    };
    while (ok && block >= 0) {
      uint32_t unit, h;
      magic_divmod(static_cast<uint32_t>(block), a.div_hk, unit, h);
      PromptUnit w = find_unit(a, unit, narrow, place);
      if (w.tokens > 0) {  // (blocks past the last unit hold nothing)
        w.h = static_cast<int>(h);
        if (KIND == kPrCut) cut_unit(a, w, static_cast<int>(cluster_ctarank()));
        shape_unit<KIND>(a, w, turn);
        turn ^= w.nb & 1;
        publish(w);
        if (!ok) break;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || w.nb == 0 || (w.split ? t != 0 : w.blocks[t] == 0)) continue;
          // (the last products that read this tile of Q are done)
          if (q_uses[t] > 0 && !(ok = warp_wait(q_empty(t), (q_uses[t] - 1) & 1, limit, abort_flag))) continue;
          if (lane == 0) {
            mbar_arrive_expect_tx(q_full(t), static_cast<uint32_t>(a.tok * a.group) * 128u * (D / 64));
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(base + C::Q_OFF + t * C::TILE + c * C::CHUNK, &a.tm_q, q_full(t), c * 64, w.h * a.group,
                          w.row0 + t * a.tok);
          }
          __syncwarp();
          ++q_uses[t];
        }
        if (!ok) break;
        if (KIND == kPrCut) break;  // (a cluster has one unit)
        // (as long as the unit is: 10 us a block of keys besides the limit)
        if (!(ok = warp_wait(near_end, (it - 1) & 1, limit + static_cast<uint64_t>(w.nb) * 10000u, abort_flag))) break;
      }
      if (KIND == kPrCut) break;
      // the next one (a CTA is at most one ahead of itself: the second of two
      // places is free when the unit before the last is done)
      if (lane == 0) {
        mbar_arrive_expect_tx(taken, 16);
        take_block(base + C::TAKEN_OFF, taken);
      }
      ++asked;
      if (!(ok = warp_wait(taken, (asked - 1) & 1, limit, abort_flag))) break;
      block = taken_block(base + C::TAKEN_OFF);
      fence_proxy_async_smem();  // (read before the next answer is written)
      __syncwarp();
    }
    if (ok) {
      PromptUnit w{};
      w.tokens = -1;
      publish(w);
    }
    if (!ok && lane == 0 && !*abort_flag) prompt_timeout(a, abort_flag, 4);
  } else {
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;  // this warp's tensor-memory lanes
    const uint32_t s_addr = tmem + lanes + t * C::S_COL;
    const uint32_t p_addr = tmem + lanes + C::P_COL + t * C::P_STEP;
    const uint32_t o_addr = tmem + lanes + C::O_COL + t * D;
    uint32_t tok, g;
    magic_divmod(static_cast<uint32_t>(row), a.div_group, tok, g);
    bool ok = true;
    int s_uses = 0, o_uses = 0, joins = 0;
    for (int it = 0; ok; ++it) {
      if (!(ok = unit_ready(it))) break;
      const PromptUnit* w = &units[it & 1];
      if (w->tokens < 0) break;
      const int my_blocks = w->blocks[t], split = KIND != kPrMany ? w->split : 0;
      const bool live = static_cast<int>(tok) < w->toks[t];
      const int my_tok = static_cast<int>(tok) + (split ? 0 : t * a.tok);
      const int vis = a.causal ? min(my_tok + w->shift + 1, w->nk) : w->nk;
      // keys of the tile's first block, and between its blocks
      const int key0 = split ? (t ^ w->start) * kPrKeys : 0, key_step = split ? 2 * kPrKeys : kPrKeys;
      float m = -INFINITY, l = 0.0f;
      for (int j = 0; j < my_blocks; ++j, ++s_uses) {
        if (!(ok = warp_wait(s_full(t), s_uses & 1, limit, abort_flag))) break;
        tc_fence_after();
        // The first half of P against the reference as it stands (the first
        // block's maximum), while the block's maximum is found; in the rare
        // block that exceeds the reference by 2^kPrLazy in some row, the
        // reference moves and the half is made again.
        const int valid = vis - key0 - j * key_step;
        const bool masked = __any_sync(0xffffffffu, valid < kPrKeys);
        const float2 cs2 = make_float2(a.cs, a.cs);
        float2 sum[4];
        uint32_t sv[128], pk[32];
        bool known = j > 0;  // whether there is a reference to go by
        // (the block before has been added to O, and the second half of its P
        // read; with P over S that is so once S is there)
        bool added = !kApart || j == 0;
        auto wait_added = [&] {
          if (!added && ok) {
            ok = warp_wait(o_full(t), (o_uses + j - 1) & 1, limit, abort_flag);
            tc_fence_after();
          }
          added = true;
          return ok;
        };
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
          if (!known) {
            known = true;
            float mp[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) mp[u] = __uint_as_float(sv[u]);
#pragma unroll
            for (int i = 4; i < 128; i += 4)
              mp[(i >> 2) & 3] = max3(mp[(i >> 2) & 3], fmaxf(__uint_as_float(sv[i]), __uint_as_float(sv[i + 1])),
                                      fmaxf(__uint_as_float(sv[i + 2]), __uint_as_float(sv[i + 3])));
            m = fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3])) * a.cs;
            if (!(m > -INFINITY)) m = -INFINITY;  // (nothing but NaN)
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
            // (P over S: the product before has completed, since this S was
            // issued after it by the same thread, and its barrier covers all
            // that was issued before)
            if (!wait_added()) break;
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
        if (!ok) break;
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
        if (!wait_added()) break;
        st_tmem_x32(p_addr + 32u, pk);
        st_tmem_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(t, 1));
        const float2 s4 = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
        l += s4.x + s4.y;
      }
      if (ok && my_blocks > 0) {
        if (kApart) o_uses += my_blocks - 1;
        ok = warp_wait(o_full(t), o_uses & 1, limit, abort_flag);
        ++o_uses;
      }
      // f0, f1: what the tiles' sums are multiplied by (f1 only where two are
      // joined), 0 for one that has none
      float f0 = l == 0.0f ? 0.0f : 1.0f / l, f1 = 0.0f, top = m;
      bool use0 = my_blocks > 0, use1 = false;
      uint32_t o0 = o_addr, o1 = o_addr;
      int c0 = 0, c1 = D;
      if (split) {
        // The warp of the other tile has the same rows: the two exchange their
        // {m, l} and each writes half of the columns.
        const int q = warp & 3;
        const uint32_t xch = base + C::XCH_OFF + row * 8;
        st_shared_f32(xch + t * kPrRows * 8, m);
        st_shared_f32(xch + t * kPrRows * 8 + 4, l);
        tc_fence_before();
        __syncwarp();
        if (ok) {
          if (lane == 0) mbar_arrive(join_ready(t, q));
          ok = warp_wait(join_ready(t ^ 1, q), joins & 1, limit, abort_flag);
        }
        if (ok) {
          // (products and sums rounded each by itself, so that it is the same
          // whichever tile is which: that depends on what the CTA had before)
          const float om = ld_shared_f32(xch + (t ^ 1) * kPrRows * 8), ol = ld_shared_f32(xch + (t ^ 1) * kPrRows * 8 + 4);
          top = fmaxf(m, om);
          const float ref = top == -INFINITY ? 0.0f : top;
          const float g0 = ex2(m - ref), g1 = ex2(om - ref);
          l = __fadd_rn(__fmul_rn(l, g0), __fmul_rn(ol, g1));
          const float inv = KIND == kPrCut ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
          f0 = g0 * inv;
          f1 = g1 * inv;
          use1 = w->blocks[t ^ 1] > 0;
          o1 = tmem + lanes + C::O_COL + (t ^ 1) * D;
          c0 = t * (D / 2);
          c1 = c0 + D / 2;
        }
      }
      if (!ok) break;
      tc_fence_after();
      if constexpr (KIND == kPrCut) {
        // The part's sums go where the ring was (nothing reads it any more:
        // both tiles' last products are done).
        if (t == 0) {
          st_shared_f32(base + C::PART_ML_OFF + row * 8, top);
          st_shared_f32(base + C::PART_ML_OFF + row * 8 + 4, l);
        }
#pragma unroll 1
        for (int c = c0; c < c1; c += 32) {
          uint32_t v[32], u[32];
          if (use0) {
            tc_ld_32x32b_x32(o0 + c, v);
            tc_wait_ld_regs(v);
          }
          if (use1) {
            tc_ld_32x32b_x32(o1 + c, u);
            tc_wait_ld_regs(u);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float x = use0 ? __fmul_rn(__uint_as_float(v[i]), f0) : 0.0f;
            v[i] = __float_as_uint(use1 ? __fadd_rn(__fmul_rn(__uint_as_float(u[i]), f1), x) : x);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            st_shared_v4(base + C::PART_OFF + (c / 4 + i) * C::PART_STEP + row * 16, v[4 * i], v[4 * i + 1], v[4 * i + 2],
                         v[4 * i + 3]);
        }
        tc_fence_before();
        break;
      }
      const bool odd = *const_cast<volatile int*>(&w->odd) != 0;  // (set before the last product was let go)
      // Four lanes exchange 16-byte pieces of their rows, so that a store
      // writes 64 bytes of each of eight rows (a row a lane, 16 bytes of 32
      // rows a store, took 5,500 cycles a unit).
      const int64_t at = live ? static_cast<int64_t>(w->row0 + my_tok) * a.os +
                                    static_cast<int64_t>(w->h * a.group + static_cast<int>(g)) * D
                              : -1;
      int64_t row_at[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) row_at[k] = __shfl_sync(0xffffffffu, at, (lane & ~3) + k);
#pragma unroll 1
      for (int c = c0; c < c1; c += 32) {
        uint32_t v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0u;
        if (use0) {
          tc_ld_32x32b_x32(o0 + c, v);
          tc_wait_ld_regs(v);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__fmul_rn(__uint_as_float(v[i]), f0));
        }
        if (use1) {
          uint32_t u[32];
          tc_ld_32x32b_x32(o1 + c, u);
          tc_wait_ld_regs(u);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            v[i] = __float_as_uint(__fadd_rn(__fmul_rn(__uint_as_float(u[i]), f1), __uint_as_float(v[i])));
        }
        if (odd && live) {
#pragma unroll 1
          for (int k = w->all_see; k < vis; ++k)
            add_odd<BF16>(a.v + static_cast<int64_t>(w->key_row + k) * a.vs + w->h * D + c, v);
        }
        uint32_t y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          y[i] = l == 0.0f ? 0u : pack_pair16<BF16>(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
        exchange4(y, lane);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (row_at[k] >= 0)
            st_global_v4(a.out + row_at[k] + c + (lane & 3) * 8, y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
      }
      tc_fence_before();
      __syncwarp();
      if (split) {
        // (the other warp has read this tile's sums too, before they are written again)
        if (lane == 0) mbar_arrive(join_done(t, warp & 3));
        if (!(ok = warp_wait(join_done(t ^ 1, warp & 3), joins & 1, limit, abort_flag))) break;
        ++joins;
      }
      if (lane == 0) mbar_arrive(unit_empty(it & 1));
    }
    if (!ok && lane == 0) prompt_timeout(a, abort_flag, 2);
  }

  // ------------------------------------------------------------ teardown
  __syncthreads();
  const uint64_t drain = drain_ns(limit);
  if ((warp == 8 || warp == 10) && *abort_flag) {
    // let the loads still in flight land before the CTA exits
    volatile int no_abort = 0;
    const int which = warp == 10;
    for (uint32_t n = issued > C::TURNS ? issued - C::TURNS : 0u; n < issued; ++n)
      if (!withheld(which, n)) mbar_wait_bounded(full(2 * (n % C::TURNS) + which), n / C::TURNS & 1, drain, &no_abort);
  }
  if (warp == 11 && *abort_flag) {
    volatile int no_abort = 0;
    for (int t = 0; t < 2; ++t)
      if (q_uses[t] > 0) mbar_wait_bounded(q_full(t), (q_uses[t] - 1) & 1, drain, &no_abort);
    if (asked > 0) mbar_wait_bounded(taken, (asked - 1) & 1, drain, &no_abort);
  }
  if (warp == 9) {
    volatile int no_abort = 0;
    mbar_wait_bounded(teardown, 0, drain, &no_abort);
  }
  if constexpr (KIND == kPrCut) {
    // (every thread of the cluster comes here, whether its waits ran out or
    // not; a unit's geometry is written without a wait)
    __syncwarp();
    cluster_sync_all();
    if (units[0].tokens > 0) {
      const uint32_t rank = cluster_ctarank();
      static_assert(kPrParts == 8, "2, 4 or 8 parts");
      if (a.lg_parts == 1)
        join_parts<D, BF16, 1>(a, units[0], base, rank);
      else if (a.lg_parts == 2)
        join_parts<D, BF16, 2>(a, units[0], base, rank);
      else
        join_parts<D, BF16, 3>(a, units[0], base, rank);
    }
    __syncwarp();
    cluster_sync_all();  // the parts have been read
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

template <int D, bool BF16, PromptKind KIND>
cudaError_t launch_prompt_as(const PromptArgs& a, unsigned grid, cudaStream_t stream) {
  using C = PromptCfg<D, KIND>;
  const cudaError_t e = set_smem_once<prompt_kernel<D, BF16, KIND>>(static_cast<int>(C::SMEM));
  if (e != cudaSuccess) return e;
  if (KIND == kPrCut)
    return launch_pdl_cluster(prompt_kernel<D, BF16, KIND>, dim3(grid), dim3(kPrThreads), C::SMEM, stream, 1u << a.lg_parts, a);
  return launch_pdl(prompt_kernel<D, BF16, KIND>, dim3(grid), dim3(kPrThreads), C::SMEM, stream, a);
}

template <int D, bool BF16>
cudaError_t launch_prompt(const PromptArgs& a, PromptKind kind, unsigned grid, cudaStream_t stream) {
  return kind == kPrCut   ? launch_prompt_as<D, BF16, kPrCut>(a, grid, stream)
         : kind == kPrFew ? launch_prompt_as<D, BF16, kPrFew>(a, grid, stream)
                          : launch_prompt_as<D, BF16, kPrMany>(a, grid, stream);
}

// CTAs that run at once in clusters of `parts` CTAs (of a whole number of
// which a group of SMs has room); < 0: an error.
template <int D, bool BF16>
int resident_ctas(unsigned parts) {
  using C = PromptCfg<D, kPrCut>;
  if (set_smem_once<prompt_kernel<D, BF16, kPrCut>>(static_cast<int>(C::SMEM)) != cudaSuccess) return -1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(parts);
  cfg.blockDim = dim3(kPrThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {parts, 1, 1};
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, prompt_kernel<D, BF16, kPrCut>, &cfg) != cudaSuccess) return -1;
  return n * static_cast<int>(parts);
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
  int device = -1;
  int resident[3] = {0, 0, 0};  // CTAs that run at once in clusters of 2, 4, 8
  lgt::DeviceStatus* d_status = nullptr;
  uint64_t wait_limit_ns = 0;
  int withhold_armed = 0;  // attn_prompt_withhold_load: the next run withholds a load (one shot)
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
  p->device = dev;
  p->wait_limit_ns = lgt::prompt_wait_limit();
  if (cudaMalloc(&p->d_status, 16) != cudaSuccess || cudaMemset(p->d_status, 0, 16) != cudaSuccess) {
    cudaGetLastError();
    if (p->d_status) cudaFree(p->d_status);
    delete p;
    return GEMM_ERR_CUDA;
  }
  for (int i = 0; i < 3; ++i) {
    const bool bf16 = d.dtype == GEMM_BF16;
    p->resident[i] = d.head_dim == 128 ? (bf16 ? lgt::resident_ctas<128, true>(2u << i) : lgt::resident_ctas<128, false>(2u << i))
                                       : (bf16 ? lgt::resident_ctas<64, true>(2u << i) : lgt::resident_ctas<64, false>(2u << i));
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
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  if (dev != plan->device) return GEMM_ERR_INVALID_ARG;  // (the status word is there)
  // Units of `span` tokens, at most: what is past the last one is found out by the CTAs.
  const int64_t seqs = std::min<int64_t>(batch, total_q);
  auto units_of = [&](int64_t span) { return (total_q + seqs * (span - 1)) / span * d.k_heads; };
  const int64_t narrow = units_of(tok), blocks = total_k / lgt::kPrKeys / seqs;
  int lg = 0;
  for (int i = 1; i <= 3; ++i)
    if (narrow << i <= plan->resident[i - 1] && blocks - (blocks >> i) >= lgt::kPrSpare) lg = i;
  const lgt::PromptKind kind = lg > 0                                                         ? lgt::kPrCut
                               : units_of(2 * tok) < static_cast<int64_t>(lgt::kPrFill) * sms ? lgt::kPrFew
                                                                                              : lgt::kPrMany;
  const int64_t units = kind == lgt::kPrMany ? units_of(2 * tok) : narrow << lg;
  if (total_q > (int64_t{1} << 30) || total_k > (int64_t{1} << 30) || units >= (int64_t{1} << 31) || batch > lgt::kPrMaxBatch)
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
  a.lg_parts = lg;
  a.withhold = plan->withhold_armed ? __atomic_exchange_n(&plan->withhold_armed, 0, __ATOMIC_ACQ_REL) : 0;
  a.div_hk = lgt::magic_encode(static_cast<uint32_t>(d.k_heads));
  a.div_group = lgt::magic_encode(static_cast<uint32_t>(group));
  a.sms = sms;
  a.div_tok = lgt::magic_encode(static_cast<uint32_t>(tok));
  a.div_pair = lgt::magic_encode(static_cast<uint32_t>(2 * tok));
  a.cs = (d.scale > 0.0f ? d.scale : 1.0f / std::sqrt(static_cast<float>(d.head_dim))) * 1.4426950408889634f;
  const bool bf16 = d.dtype == GEMM_BF16;
  a.idesc_s = lgt::idesc_f16(bf16, 0u, 0u, lgt::kPrRows, lgt::kPrKeys);
  a.idesc_pv = lgt::idesc_f16(bf16, 0u, 1u, lgt::kPrRows, static_cast<uint32_t>(d.head_dim));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned grid = static_cast<unsigned>(units);
  const cudaError_t e = d.head_dim == 128
                            ? (bf16 ? lgt::launch_prompt<128, true>(a, kind, grid, s) : lgt::launch_prompt<128, false>(a, kind, grid, s))
                            : (bf16 ? lgt::launch_prompt<64, true>(a, kind, grid, s) : lgt::launch_prompt<64, false>(a, kind, grid, s));
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

gemm_status_t attn_prompt_withhold_load(attn_prompt_plan_t* plan) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  __atomic_store_n(&plan->withhold_armed, 1, __ATOMIC_RELEASE);
  return GEMM_OK;
}

gemm_status_t attn_prompt_destroy(attn_prompt_plan_t* plan) {
  if (!plan) return GEMM_OK;
  if (plan->d_status) cudaFree(plan->d_status);
  delete plan;
  return GEMM_OK;
}

}  // extern "C"
