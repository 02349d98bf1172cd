// Norm and position rotation of queries and keys in one pass
// (include/attn_rope.h).
//
// A head's d values belong to a group of LG lanes (the least power of two
// with LG * 8 >= d), eight values a lane: in the half layout two runs of
// four, [4u, 4u + 4) of the first half of the rotated part and the same of
// the second, so that both values of each of the lane's four pairs are its
// own; otherwise eight neighbours.  The head's sum of squares goes around
// the group by a shuffle butterfly; everything is fp32 and is rounded once.
//
// The angle.  f_i / (2 pi), the turns a position, is held as a 64-bit binary
// fraction.  position * fraction modulo 2^64 is the phase modulo one turn,
// exactly: integer multiplication wraps where the angle does.  So the angle
// is right to 2^-53 of a turn times the position whatever the position is,
// with no table to read and no argument reduction; the sine and cosine are
// taken of an angle in [-pi, pi], where the hardware's approximations are
// within 2^-20.9 absolute, a thousandth of an fp16 rounding.
//
// Bound: memory, each value read and written once.  A group takes kItems
// neighbouring heads and loads all of them before it works on the first
// (16 bytes a lane each), and computes the sines again only where the token
// changes.
#include <cmath>
#include <cstdint>
#include <new>

#include "attn_rope.h"
#include "half_types.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace lgt {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = 128;  // head_dim 256

struct RopeArgs {
  const uint16_t *q, *k, *wq, *wk;
  uint16_t *qo, *ko;
  const int32_t* pos;
  int64_t qs, ks, qos, kos;
  uint32_t items;  // tokens * heads
  MagicDiv div_heads;
  int32_t hq, d, rot;
  float eps, inv_d, magnitude;
  uint64_t turns[kRopeMaxPairs];  // of pair i a position, as a fraction of 2^64
};

// One lane's part of one head: where its two runs of four values are.
template <bool HALF>
__device__ __forceinline__ void run_offsets(int u, int rot, int& o0, int& o1) {
  if (HALF && 8 * u < rot) {
    o0 = 4 * u;
    o1 = rot / 2 + 4 * u;
  } else {
    o0 = 8 * u;
    o1 = 8 * u + 4;
  }
}

template <int LG, bool BF16, bool HALF, int ITEMS>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int u = threadIdx.x % LG;
  const uint32_t first = (blockIdx.x * (kRopeThreads / LG) + threadIdx.x / LG) * ITEMS;
  const bool mine = 8 * u < a.d;
  const bool turned = 8 * u < a.rot;
  const bool norms = a.wq != nullptr || a.wk != nullptr;
  int o0, o1;
  run_offsets<HALF>(u, a.rot, o0, o1);

  uint2 x0[ITEMS], x1[ITEMS];
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    x0[j] = x1[j] = make_uint2(0u, 0u);
    if (first + j < a.items && mine) {
      uint32_t t, h;
      magic_divmod(first + j, a.div_heads, t, h);
      const bool is_q = h < static_cast<uint32_t>(a.hq);
      const uint16_t* src = is_q ? a.q + static_cast<int64_t>(t) * a.qs + static_cast<int64_t>(h) * a.d
                                 : a.k + static_cast<int64_t>(t) * a.ks + static_cast<int64_t>(h - a.hq) * a.d;
      if constexpr (HALF) {
        x0[j] = ld_stream_v2(src + o0);
        x1[j] = ld_stream_v2(src + o1);
      } else {
        const uint4 v = ld_stream_v4(src + o0);
        x0[j] = make_uint2(v.x, v.y);
        x1[j] = make_uint2(v.z, v.w);
      }
    }
  }

  float cs[4], sn[4], w[8];
  uint32_t have_t = 0xffffffffu;
  int have_w = -1;
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    uint32_t t, h;
    magic_divmod(first + j < a.items ? first + j : a.items - 1, a.div_heads, t, h);
    const bool is_q = h < static_cast<uint32_t>(a.hq);
    float y[8];
    {
      const float2 p0 = unpack_pair16<BF16>(x0[j].x), p1 = unpack_pair16<BF16>(x0[j].y);
      const float2 p2 = unpack_pair16<BF16>(x1[j].x), p3 = unpack_pair16<BF16>(x1[j].y);
      y[0] = p0.x; y[1] = p0.y; y[2] = p1.x; y[3] = p1.y;
      y[4] = p2.x; y[5] = p2.y; y[6] = p3.x; y[7] = p3.y;
    }
    const uint16_t* wt = is_q ? a.wq : a.wk;
    if (norms) {  // (the same for every lane: the groups of a warp may be at heads with and without a norm)
      float ss = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
      for (int o = LG / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (wt && mine) {
        const float r = rsqrtf(fmaf(ss, a.inv_d, a.eps));
        if (have_w != static_cast<int>(is_q)) {
          have_w = is_q;
          const uint2 w0 = *reinterpret_cast<const uint2*>(wt + o0), w1 = *reinterpret_cast<const uint2*>(wt + o1);
          const float2 p0 = unpack_pair16<BF16>(w0.x), p1 = unpack_pair16<BF16>(w0.y);
          const float2 p2 = unpack_pair16<BF16>(w1.x), p3 = unpack_pair16<BF16>(w1.y);
          w[0] = p0.x; w[1] = p0.y; w[2] = p1.x; w[3] = p1.y;
          w[4] = p2.x; w[5] = p2.y; w[6] = p3.x; w[7] = p3.y;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = y[e] * r * w[e];
      }
    }
    if (turned) {
      if (t != have_t) {
        have_t = t;
        const uint64_t p = static_cast<uint64_t>(static_cast<int64_t>(a.pos[t]));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint64_t phase = p * a.turns[4 * u + e];
          const float ang = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
          sn[e] = __sinf(ang) * a.magnitude;
          cs[e] = __cosf(ang) * a.magnitude;
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float& lo = HALF ? y[e] : y[2 * e];
        float& hi = HALF ? y[4 + e] : y[2 * e + 1];
        const float c = lo * cs[e] - hi * sn[e], s = hi * cs[e] + lo * sn[e];
        lo = c;
        hi = s;
      }
    }
    if (first + j < a.items && mine) {
      uint16_t* dst = is_q ? a.qo + static_cast<int64_t>(t) * a.qos + static_cast<int64_t>(h) * a.d
                           : a.ko + static_cast<int64_t>(t) * a.kos + static_cast<int64_t>(h - a.hq) * a.d;
      const uint32_t p0 = pack_pair16<BF16>(y[0], y[1]), p1 = pack_pair16<BF16>(y[2], y[3]);
      const uint32_t p2 = pack_pair16<BF16>(y[4], y[5]), p3 = pack_pair16<BF16>(y[6], y[7]);
      if constexpr (HALF) {
        st_global_v2(dst + o0, p0, p1);
        st_global_v2(dst + o1, p2, p3);
      } else {
        st_global_v4(dst + o0, p0, p1, p2, p3);
      }
    }
  }
}

template <int LG, bool BF16, bool HALF>
cudaError_t launch_rope(const RopeArgs& a, int sms, cudaStream_t stream) {
  constexpr uint32_t groups = kRopeThreads / LG;
  // four heads a group where that still gives every SM two blocks of them
  if (a.items >= groups * 4u * 2u * static_cast<uint32_t>(sms)) {
    const uint32_t blocks = (a.items + groups * 4u - 1u) / (groups * 4u);
    return launch_pdl(rope_kernel<LG, BF16, HALF, 4>, dim3(blocks), dim3(kRopeThreads), 0, stream, a);
  }
  const uint32_t blocks = (a.items + groups - 1u) / groups;
  return launch_pdl(rope_kernel<LG, BF16, HALF, 1>, dim3(blocks), dim3(kRopeThreads), 0, stream, a);
}

template <bool BF16, bool HALF>
cudaError_t launch_rope_lg(const RopeArgs& a, int sms, cudaStream_t stream) {
  if (a.d <= 8) return launch_rope<1, BF16, HALF>(a, sms, stream);
  if (a.d <= 16) return launch_rope<2, BF16, HALF>(a, sms, stream);
  if (a.d <= 32) return launch_rope<4, BF16, HALF>(a, sms, stream);
  if (a.d <= 64) return launch_rope<8, BF16, HALF>(a, sms, stream);
  if (a.d <= 128) return launch_rope<16, BF16, HALF>(a, sms, stream);
  return launch_rope<32, BF16, HALF>(a, sms, stream);
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
