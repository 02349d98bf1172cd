// Norm and position rotation of queries and keys in one pass
// (include/attn_rope.h).
//
// A head's d values belong to a group of LG lanes, two runs of R = 8 (16
// bytes) or 4 values a lane: in the half layout R of the first half of the
// rotated part and the same R of the second, so that both values of each of
// the lane's R pairs are its own; otherwise 2R neighbours.  LG is the least
// power of two with LG * 2R >= d.  R is 8 where rot_dim and d are multiples of
// 16, which all common sizes are.  The head's sum of squares goes around the
// group by a shuffle butterfly; everything is fp32 and is rounded once.
//
// The angle.  f_i / (2 pi), the turns a position, is held as a 64-bit binary
// fraction.  position * fraction modulo 2^64 is the phase modulo one turn,
// exactly: integer multiplication wraps where the angle does.  So the angle
// is right to 2^-53 of a turn times the position whatever the position is,
// with no table to read and no argument reduction; the sine and cosine are
// taken of an angle in [-pi, pi], where the hardware's approximations are
// within 2^-20.9 absolute, a thousandth of an fp16 rounding.
//
// Bound: memory, each value read and written once.  A warp takes a chunk of
// neighbouring heads, its groups every G-th of them (or a run each, where a
// token has so few heads that the sines would be taken every few steps), two on
// their way a group; the sines are computed again only where the token changes;
// the blocks are one wave of what the registers hold.
// Measured (16384 tokens, 32 + 8 heads of 128, bf16): 55.3 us, 6.07 TB/s, 89 %
// of a copy's rate (without any arithmetic it takes as long).  A run a group
// 57.4, with loads that are not kept in L1 and plain stores 58.7; every
// sixteenth of a block's heads 62; three heads on their way with five blocks 55,
// but 1000 tokens 7.6 against 6.9; runs of four values 84, one head on its way
// 84, a ring in shared memory 63.  64 tokens: 3.8 us in a graph over three sets of
// inputs.
#include <cmath>
#include <cstdint>
#include <new>

#include "attn_rope.h"
#include "half_types.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace lgt {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeMaxPairs = 128;  // head_dim 256
constexpr uint32_t kRopeBlocks = 6;   // blocks an SM the chunks are cut for: what its registers hold (R = 8)
constexpr uint32_t kRopeBlocks4 = 9;  // the same for R = 4 (4000 tokens, 40 heads of 96, 40 turned: 18.5 us, with six 24.6)
constexpr int kRopeDepth = 2;        // heads of a group on their way

struct RopeArgs {
  const uint16_t *q, *k, *wq, *wk;
  uint16_t *qo, *ko;
  const int32_t* pos;
  int64_t qs, ks, qos, kos;
  uint32_t items;  // tokens * heads
  uint32_t chunk;  // of a group
  uint32_t stride;  // between the heads of a group
  MagicDiv div_heads;
  int32_t hq, heads, d, rot;
  float eps, inv_d, magnitude;
  uint64_t turns[kRopeMaxPairs];  // of pair i a position, as a fraction of 2^64
};

template <int R>
struct Run {  // R 16-bit values
  uint32_t w[R / 2];
};

template <int R>
__device__ __forceinline__ Run<R> load_run(const uint16_t* p) {
  Run<R> r;
  if constexpr (R == 8) {
    const uint4 v = ld_stream_v4(p);
    r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
  } else {
    const uint2 v = ld_stream_v2(p);
    r.w[0] = v.x; r.w[1] = v.y;
  }
  return r;
}

template <int R>
__device__ __forceinline__ void store_run(uint16_t* p, const Run<R>& r) {
  if constexpr (R == 8)
    st_stream_v4(p, r.w[0], r.w[1], r.w[2], r.w[3]);
  else
    st_stream_v2(p, r.w[0], r.w[1]);
}

template <int R, bool BF16>
__device__ __forceinline__ void widen_run(const Run<R>& r, float* x) {
#pragma unroll
  for (int i = 0; i < R / 2; ++i) {
    const float2 p = unpack_pair16<BF16>(r.w[i]);
    x[2 * i] = p.x;
    x[2 * i + 1] = p.y;
  }
}

template <int R, bool BF16>
__device__ __forceinline__ Run<R> narrow_run(const float* x) {
  Run<R> r;
#pragma unroll
  for (int i = 0; i < R / 2; ++i) r.w[i] = pack_pair16<BF16>(x[2 * i], x[2 * i + 1]);
  return r;
}

template <int R, int LG, bool BF16, bool HALF>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  pdl_launch_dependents();
  const int u = threadIdx.x % LG;
  constexpr uint32_t G = 32 / LG;  // groups of a warp
  const uint32_t warp = blockIdx.x * (kRopeThreads / 32) + threadIdx.x / 32, in_warp = threadIdx.x % 32 / LG;
  const uint32_t begin = min(warp * G * a.chunk, a.items), stop = min(begin + G * a.chunk, a.items);
  const uint32_t first = a.stride == 1 ? min(begin + in_warp * a.chunk, stop) : begin + in_warp;
  const uint32_t end = a.stride == 1 ? min(first + a.chunk, stop) : stop;
  const bool mine = 2 * R * u < a.d;
  const bool turned = 2 * R * u < a.rot;
  const bool norms = a.wq != nullptr || a.wk != nullptr;
  const int o0 = HALF && turned ? R * u : 2 * R * u, o1 = HALF && turned ? a.rot / 2 + R * u : 2 * R * u + R;
  auto is_query = [&](uint32_t hh) { return hh < static_cast<uint32_t>(a.hq); };
  pdl_wait();

  // two heads on their way; the place of one is loaded again as soon as it is taken
  Run<R> x0[kRopeDepth], x1[kRopeDepth];
  uint32_t lt[kRopeDepth], lh[kRopeDepth];
  auto load = [&](int j, uint32_t item) {
    if (item < end) {
      magic_divmod(item, a.div_heads, lt[j], lh[j]);
      const uint32_t t = lt[j], h = lh[j];
      if (mine) {
        const uint16_t* src = is_query(h) ? a.q + static_cast<int64_t>(t) * a.qs + h * a.d
                                          : a.k + static_cast<int64_t>(t) * a.ks + (h - a.hq) * a.d;
        x0[j] = load_run<R>(src + o0);
        x1[j] = load_run<R>(src + o1);
      }
    }
  };
#pragma unroll
  for (int j = 0; j < kRopeDepth; ++j) {
#pragma unroll
    for (int i = 0; i < R / 2; ++i) x0[j].w[i] = x1[j].w[i] = 0u;
    lt[j] = lh[j] = 0u;
    load(j, first + j * a.stride);
  }

  float cs[R], sn[R];
  Run<R> w0, w1;
  uint32_t have_t = 0xffffffffu;
  int have_w = -1;
  // (every lane of a warp goes round as often: the butterflies are of all)
  for (uint32_t step = 0; step < a.chunk; step += kRopeDepth) {
#pragma unroll
    for (int j = 0; j < kRopeDepth; ++j) {
      const uint32_t item = first + (step + j) * a.stride;
      const uint32_t ct = lt[j], ch = lh[j];
      const bool is_q = is_query(ch);
      float y[2 * R];
      widen_run<R, BF16>(x0[j], y);
      widen_run<R, BF16>(x1[j], y + R);
      load(j, item + kRopeDepth * a.stride);
      if (norms) {
        float ss[2] = {};
#pragma unroll
        for (int e = 0; e < 2 * R; ++e) ss[e & 1] = fmaf(y[e], y[e], ss[e & 1]);
        ss[0] += ss[1];
#pragma unroll
        for (int o = LG / 2; o > 0; o >>= 1) ss[0] += __shfl_xor_sync(0xffffffffu, ss[0], o);
        const uint16_t* wt = is_q ? a.wq : a.wk;
        if (wt && mine) {
          const float r = rsqrtf(fmaf(ss[0], a.inv_d, a.eps));
          if (have_w != static_cast<int>(is_q)) {
            have_w = is_q;
#pragma unroll
            for (int i = 0; i < R / 2; ++i) {
              w0.w[i] = __ldg(reinterpret_cast<const uint32_t*>(wt + o0) + i);
              w1.w[i] = __ldg(reinterpret_cast<const uint32_t*>(wt + o1) + i);
            }
          }
          float w[2 * R];
          widen_run<R, BF16>(w0, w);
          widen_run<R, BF16>(w1, w + R);
#pragma unroll
          for (int e = 0; e < 2 * R; ++e) y[e] = y[e] * r * w[e];
        }
      }
      if (turned) {
        if (ct != have_t && item < end) {
          have_t = ct;
          const int32_t p = __ldg(a.pos + ct);
#pragma unroll
          for (int e = 0; e < R; ++e) {
            // bits 32 .. 63 of position * turns
            const uint64_t f = a.turns[R * u + e];
            const uint32_t lo = static_cast<uint32_t>(f), hi = static_cast<uint32_t>(f >> 32);
            const uint32_t phase = __umulhi(static_cast<uint32_t>(p), lo) + static_cast<uint32_t>(p) * hi - (p < 0 ? lo : 0u);
            const float ang = static_cast<float>(static_cast<int32_t>(phase)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
            sn[e] = __sinf(ang) * a.magnitude;
            cs[e] = __cosf(ang) * a.magnitude;
          }
        }
#pragma unroll
        for (int e = 0; e < R; ++e) {
          float& lo = HALF ? y[e] : y[2 * e];
          float& hi = HALF ? y[R + e] : y[2 * e + 1];
          const float c = lo * cs[e] - hi * sn[e], s = hi * cs[e] + lo * sn[e];
          lo = c;
          hi = s;
        }
      }
      if (item < end && mine) {
        uint16_t* dst = is_q ? a.qo + static_cast<int64_t>(ct) * a.qos + ch * a.d
                             : a.ko + static_cast<int64_t>(ct) * a.kos + (ch - a.hq) * a.d;
        store_run<R>(dst + o0, narrow_run<R, BF16>(y));
        store_run<R>(dst + o1, narrow_run<R, BF16>(y + R));
      }
    }
  }
}

template <int R, int LG, bool BF16, bool HALF>
cudaError_t launch_rope(RopeArgs& a, int sms, cudaStream_t stream) {
  constexpr uint32_t groups = kRopeThreads / LG;
  // Chunks that give every SM kRopeBlocks blocks, whole pairs of heads; one
  // head a group where there are fewer than that.
  const uint32_t most = static_cast<uint32_t>(sms) * (R == 8 ? kRopeBlocks : kRopeBlocks4) * groups;
  a.chunk = (a.items + most - 1u) / most;
  // (16384 tokens, us a run a group and interleaved: 8 + 1 heads of 128, 64
  // turned, 17.6 and 19.1; 8 + 8 of 128 25.7 and 24.6; 32 + 8 of 128 58.3 and
  // 57.1; 16 + 4 of 256 60.3 and 58.0; 12 + 4 of 64 16.1 and 15.2)
  a.stride = a.heads < 16 ? 1u : 32 / LG;
  const uint32_t per_block = groups * a.chunk, blocks = a.items / per_block + (a.items % per_block ? 1u : 0u);
  return launch_pdl(rope_kernel<R, LG, BF16, HALF>, dim3(blocks), dim3(kRopeThreads), 0, stream, a);
}

template <bool BF16, bool HALF>
cudaError_t launch_rope_lg(RopeArgs& a, int sms, cudaStream_t stream) {
  if (a.d % 16 == 0 && a.rot % 16 == 0) {
    if (a.d <= 16) return launch_rope<8, 1, BF16, HALF>(a, sms, stream);
    if (a.d <= 32) return launch_rope<8, 2, BF16, HALF>(a, sms, stream);
    if (a.d <= 64) return launch_rope<8, 4, BF16, HALF>(a, sms, stream);
    if (a.d <= 128) return launch_rope<8, 8, BF16, HALF>(a, sms, stream);
    return launch_rope<8, 16, BF16, HALF>(a, sms, stream);
  }
  if (a.d <= 64) return launch_rope<4, 8, BF16, HALF>(a, sms, stream);
  if (a.d <= 128) return launch_rope<4, 16, BF16, HALF>(a, sms, stream);
  return launch_rope<4, 32, BF16, HALF>(a, sms, stream);
}

bool rope_desc_ok(const attn_rope_desc_t& d, bool own_frequencies) {
  if (d.q_heads < 1 || d.k_heads < 1 || d.head_dim < 8 || d.head_dim > 256 || d.head_dim % 8 != 0) return false;
  if (d.rot_dim < 0 || d.rot_dim > d.head_dim || d.rot_dim % 8 != 0) return false;
  if (d.layout != ATTN_ROPE_HALF && d.layout != ATTN_ROPE_INTERLEAVED) return false;
  if (d.dtype != GEMM_F16 && d.dtype != GEMM_BF16) return false;
  if (!(d.eps >= 0.0f) || !std::isfinite(d.eps) || !std::isfinite(d.magnitude)) return false;
  if (own_frequencies) return true;
  if (!(d.base > 0.0) || !std::isfinite(d.base)) return false;
  if (!(d.factor == 0.0 || (d.factor >= 1.0 && std::isfinite(d.factor)))) return false;
  if (!(d.low_turns >= 0.0) || !(d.high_turns >= d.low_turns) || !std::isfinite(d.high_turns)) return false;
  if (d.factor > 1.0 && d.high_turns > 0.0 && (!(d.context > 0.0) || !std::isfinite(d.context))) return false;
  return true;
}

constexpr double kTwoPi = 6.283185307179586476925286766559;

void rope_frequencies(const attn_rope_desc_t& d, double* f) {
  for (int i = 0; i < d.rot_dim / 2; ++i) {
    f[i] = std::pow(d.base, -2.0 * i / d.rot_dim);
    if (d.factor > 1.0) {
      double keep = 0.0;
      if (d.high_turns > 0.0) {
        const double r = d.context * f[i] / kTwoPi;
        keep = r >= d.high_turns ? 1.0 : r <= d.low_turns ? 0.0 : (r - d.low_turns) / (d.high_turns - d.low_turns);
      }
      f[i] *= keep + (1.0 - keep) / d.factor;
    }
  }
}

}  // namespace
}  // namespace lgt

struct attn_rope_plan {
  attn_rope_desc_t d;
  uint64_t turns[lgt::kRopeMaxPairs];
};

extern "C" {

gemm_status_t attn_rope_frequencies(const attn_rope_desc_t* desc, double* frequencies) {
  if (!desc || !frequencies || !lgt::rope_desc_ok(*desc, false)) return GEMM_ERR_INVALID_ARG;
  lgt::rope_frequencies(*desc, frequencies);
  return GEMM_OK;
}

gemm_status_t attn_rope_create(const attn_rope_desc_t* desc, const double* frequencies, attn_rope_plan_t** plan) {
  if (!plan) return GEMM_ERR_INVALID_ARG;
  *plan = nullptr;
  if (!desc || !lgt::rope_desc_ok(*desc, frequencies != nullptr)) return GEMM_ERR_INVALID_ARG;
  double f[lgt::kRopeMaxPairs] = {};
  const int pairs = desc->rot_dim / 2;
  if (frequencies) {
    for (int i = 0; i < pairs; ++i) {
      if (!std::isfinite(frequencies[i])) return GEMM_ERR_INVALID_ARG;
      f[i] = frequencies[i];
    }
  } else {
    lgt::rope_frequencies(*desc, f);
  }
  attn_rope_plan* p = new (std::nothrow) attn_rope_plan();
  if (!p) return GEMM_ERR_CUDA;
  p->d = *desc;
  for (int i = 0; i < pairs; ++i) {
    double turns = f[i] / lgt::kTwoPi;
    turns -= std::floor(turns);  // whole turns a position do not show
    // (just below one turn the product may round to 2^64, which is no turn)
    const double scaled = turns * 18446744073709551616.0;
    p->turns[i] = scaled >= 18446744073709551616.0 ? 0u : static_cast<uint64_t>(scaled);
  }
  *plan = p;
  return GEMM_OK;
}

gemm_status_t attn_rope_run(const attn_rope_plan_t* plan, const void* Q, int64_t q_stride, const void* K,
                            int64_t k_stride, const void* q_weight, const void* k_weight, const int32_t* positions,
                            int64_t tokens, void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                            void* stream) {
  if (!plan || tokens < 0) return GEMM_ERR_INVALID_ARG;
  const attn_rope_desc_t& d = plan->d;
  const int64_t qrow = static_cast<int64_t>(d.q_heads) * d.head_dim, krow = static_cast<int64_t>(d.k_heads) * d.head_dim;
  int64_t* strides[4] = {&q_stride, &q_out_stride, &k_stride, &k_out_stride};
  for (int i = 0; i < 4; ++i) {
    const int64_t row = i < 2 ? qrow : krow;
    if (*strides[i] == 0) *strides[i] = row;
    if (*strides[i] < row || *strides[i] % 8 != 0) return GEMM_ERR_INVALID_ARG;
  }
  if (tokens == 0) return GEMM_OK;
  if (!Q || !K || !q_out || !k_out || (!positions && d.rot_dim > 0)) return GEMM_ERR_INVALID_ARG;
  for (const void* p : {Q, K, q_weight, k_weight, static_cast<const void*>(q_out), static_cast<const void*>(k_out)})
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return GEMM_ERR_ALIGNMENT;
  if (reinterpret_cast<uintptr_t>(positions) % 4 != 0) return GEMM_ERR_ALIGNMENT;
  const int64_t heads = static_cast<int64_t>(d.q_heads) + d.k_heads;
  if (heads >= (int64_t{1} << 31) || tokens > ((int64_t{1} << 31) - 1) / heads) return GEMM_ERR_UNSUPPORTED;

  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  lgt::RopeArgs a;
  a.q = static_cast<const uint16_t*>(Q);
  a.k = static_cast<const uint16_t*>(K);
  a.wq = static_cast<const uint16_t*>(q_weight);
  a.wk = static_cast<const uint16_t*>(k_weight);
  a.qo = static_cast<uint16_t*>(q_out);
  a.ko = static_cast<uint16_t*>(k_out);
  a.pos = positions;
  a.qs = q_stride;
  a.ks = k_stride;
  a.qos = q_out_stride;
  a.kos = k_out_stride;
  a.items = static_cast<uint32_t>(tokens * heads);
  a.div_heads = lgt::magic_encode(static_cast<uint32_t>(heads));
  a.hq = d.q_heads;
  a.heads = static_cast<int32_t>(heads);
  a.d = d.head_dim;
  a.rot = d.rot_dim;
  a.eps = d.eps;
  a.inv_d = 1.0f / static_cast<float>(d.head_dim);
  a.magnitude = d.magnitude == 0.0f ? 1.0f : d.magnitude;
  for (int i = 0; i < lgt::kRopeMaxPairs; ++i) a.turns[i] = plan->turns[i];
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool half = d.layout == ATTN_ROPE_HALF;
  const cudaError_t e = d.dtype == GEMM_BF16
                            ? (half ? lgt::launch_rope_lg<true, true>(a, sms, s) : lgt::launch_rope_lg<true, false>(a, sms, s))
                            : (half ? lgt::launch_rope_lg<false, true>(a, sms, s) : lgt::launch_rope_lg<false, false>(a, sms, s));
  if (e != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  return GEMM_OK;
}

gemm_status_t attn_rope_destroy(attn_rope_plan_t* plan) {
  delete plan;
  return GEMM_OK;
}

}  // extern "C"
