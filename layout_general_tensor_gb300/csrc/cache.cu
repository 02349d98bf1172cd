// Writing keys and values into the paged 8-bit cache and reading them back
// (include/attn_cache.h).
//
// One group of head_dim / 8 lanes per token and key head, eight values of K
// and eight of V a lane (16 bytes each of the 16-bit tensors, 8 of the
// codes).  The rows' largest finite magnitudes go around the group as bit
// patterns, K's and V's in one word (for magnitudes the order of the bits is
// the order of the values), and the power of two comes out of its exponent and significand without a
// logarithm: with amax = m * 2^e, 1 <= m < 2, and 448 = 1.75 * 2^8,
// ceil(log2(amax / 448)) is e - 8, and one more when m > 1.75.
//
// A row's codes and its exponent are separate stores, which nothing orders
// against those of another group: two tokens of a call with the same slot may
// leave a mixture, so a call's slots are distinct.
//
// Bound: memory; every value is read once and every code written once.
// Measured (16384 tokens, 8 heads of 128, bf16): write and read back 30.7 us,
// 6.6 TB/s, 97 % of a copy's rate; with the maxima found in fp32 and the power
// applied as two factors the write was bound by arithmetic (35 us).
#include <cstdint>

#include "cache.h"
#include "half_types.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace lgt {
namespace {

constexpr int kCacheThreads = 256;

struct CacheArgs {
  uint8_t *k, *v, *ke, *ve;
  uint16_t *kx, *vx;  // the 16-bit tensors (read by write, written by read)
  int64_t ks, vs;
  const int32_t* slots;
  int64_t num_slots;
  uint32_t items;  // tokens * heads
  MagicDiv div_heads, div_page;
  int32_t heads, page;
};

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack_pair16<BF16>(r[i]);
    x[2 * i] = p.x;
    x[2 * i + 1] = p.y;
  }
}

// The largest finite magnitude of eight 16-bit values, as the bits of its type:
// two at a time as integers, and one by one only where that finds one that is
// not finite.
template <bool BF16>
__device__ __forceinline__ uint32_t amax16(const uint4& w) {
  constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u;
  const uint32_t r[4] = {w.x & 0x7fff7fffu, w.y & 0x7fff7fffu, w.z & 0x7fff7fffu, w.w & 0x7fff7fffu};
  const uint32_t m = __vmaxu2(__vmaxu2(r[0], r[1]), __vmaxu2(r[2], r[3]));
  uint32_t most = max(m & 0xffffu, m >> 16);
  if (most >= kInf) {
    most = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = r[i] & 0xffffu, hi = r[i] >> 16;
      most = max(most, max(lo < kInf ? lo : 0u, hi < kInf ? hi : 0u));
    }
  }
  return most;
}

// power + 127 of a row with this largest magnitude.  (A bf16 subnormal's
// exponent field is 0, and so is the clamp's outcome for it.)
template <bool BF16>
__device__ __forceinline__ int row_exponent(uint32_t amax16) {
  const uint32_t amax = BF16 ? amax16 << 16 : __float_as_uint(unpack_pair16<false>(amax16).x);
  if (amax == 0) return 127;
  const int e = static_cast<int>(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, 1);
}

// Eight values times 2^(127 - exponent) as e4m3 codes.  (The power is in
// [-120, 126], and what the product loses below fp32's range is far below half
// of the least code.)
template <bool BF16>
__device__ __forceinline__ uint2 encode8(const uint4& w, int exponent) {
  const float f = __uint_as_float(static_cast<uint32_t>(254 - exponent) << 23);
  float x[8];
  unpack8<BF16>(w, x);
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(x[2 * i + 1] * f), "f"(x[2 * i] * f));
    r[i] = c;
  }
  return make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
}

template <bool BF16>
__device__ __forceinline__ uint4 decode8(const uint2& c, int exponent) {
  // (2^-127 is a subnormal)
  const float f = __uint_as_float(exponent == 0 ? 0x00400000u : static_cast<uint32_t>(exponent) << 23);
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint16_t pair = static_cast<uint16_t>((i < 2 ? c.x : c.y) >> (16 * (i & 1)));
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(pair));
    const float2 x = unpack_pair16<false>(h);
    r[i] = pack_pair16_sat<BF16>(x.x * f, x.y * f);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Where the row of `slot` and head h starts, in rows of head_dim codes.
__device__ __forceinline__ int64_t cache_row(const CacheArgs& a, int32_t slot, uint32_t h) {
  uint32_t p, off;
  magic_divmod(static_cast<uint32_t>(slot), a.div_page, p, off);
  return (static_cast<int64_t>(p) * a.heads + h) * a.page + off;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kCacheThreads) cache_write_kernel(const __grid_constant__ CacheArgs a) {
  constexpr int LG = D / 8;
  pdl_launch_dependents();
  pdl_wait();
  const int u = threadIdx.x % LG;
  const uint32_t item = blockIdx.x * (kCacheThreads / LG) + threadIdx.x / LG;
  uint32_t t = 0, h = 0;
  int32_t slot = -1;
  uint4 kw = make_uint4(0u, 0u, 0u, 0u), vw = kw;
  if (item < a.items) {
    magic_divmod(item, a.div_heads, t, h);
    kw = ld_stream_v4(a.kx + static_cast<int64_t>(t) * a.ks + h * D + u * 8);
    vw = ld_stream_v4(a.vx + static_cast<int64_t>(t) * a.vs + h * D + u * 8);
    slot = a.slots[t];
  }
  uint32_t both = amax16<BF16>(kw) | (amax16<BF16>(vw) << 16);
#pragma unroll
  for (int o = LG / 2; o > 0; o >>= 1) {
    both = __vmaxu2(both, __shfl_xor_sync(0xffffffffu, both, o));
  }
  const uint32_t km = both & 0xffffu, vm = both >> 16;
  if (slot < 0 || slot >= a.num_slots) return;
  const int64_t row = cache_row(a, slot, h);
  const int ke = row_exponent<BF16>(km), ve = row_exponent<BF16>(vm);
  const uint2 kc = encode8<BF16>(kw, ke), vc = encode8<BF16>(vw, ve);
  st_global_v2(a.k + row * D + u * 8, kc.x, kc.y);
  st_global_v2(a.v + row * D + u * 8, vc.x, vc.y);
  if (u == 0) {
    a.ke[row] = static_cast<uint8_t>(ke);
    a.ve[row] = static_cast<uint8_t>(ve);
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(const __grid_constant__ CacheArgs a) {
  constexpr int LG = D / 8;
  pdl_launch_dependents();
  pdl_wait();
  const int u = threadIdx.x % LG;
  const uint32_t item = blockIdx.x * (kCacheThreads / LG) + threadIdx.x / LG;
  if (item >= a.items) return;
  uint32_t t, h;
  magic_divmod(item, a.div_heads, t, h);
  const int32_t slot = a.slots[t];
  uint4 kw = make_uint4(0u, 0u, 0u, 0u), vw = kw;
  if (slot >= 0 && slot < a.num_slots) {
    const int64_t row = cache_row(a, slot, h);
    const uint2 kc = ld_stream_v2(a.k + row * D + u * 8), vc = ld_stream_v2(a.v + row * D + u * 8);
    kw = decode8<BF16>(kc, a.ke[row]);
    vw = decode8<BF16>(vc, a.ve[row]);
  }
  st_global_v4(a.kx + static_cast<int64_t>(t) * a.ks + h * D + u * 8, kw.x, kw.y, kw.z, kw.w);
  st_global_v4(a.vx + static_cast<int64_t>(t) * a.vs + h * D + u * 8, vw.x, vw.y, vw.z, vw.w);
}

template <bool WRITE>
gemm_status_t run_cache(const attn_cache_t* c, const void* K, int64_t k_stride, const void* V, int64_t v_stride,
                        const int32_t* slots, int64_t tokens, int32_t dtype, void* stream) {
  if (!c || tokens < 0 || (dtype != GEMM_F16 && dtype != GEMM_BF16)) return GEMM_ERR_INVALID_ARG;
  if (!cache_ok(*c)) return GEMM_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(c->k_heads) * c->head_dim;
  if (k_stride == 0) k_stride = row;
  if (v_stride == 0) v_stride = row;
  if (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0) return GEMM_ERR_INVALID_ARG;
  if (tokens == 0) return GEMM_OK;
  if (!K || !V || !slots) return GEMM_ERR_INVALID_ARG;
  for (const void* p : {K, V, static_cast<const void*>(c->k), static_cast<const void*>(c->v)})
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return GEMM_ERR_ALIGNMENT;
  if (reinterpret_cast<uintptr_t>(slots) % 4 != 0) return GEMM_ERR_ALIGNMENT;
  if (tokens > ((int64_t{1} << 31) - 1) / c->k_heads) return GEMM_ERR_UNSUPPORTED;
  CacheArgs a;
  a.k = static_cast<uint8_t*>(c->k);
  a.v = static_cast<uint8_t*>(c->v);
  a.ke = static_cast<uint8_t*>(c->k_exp);
  a.ve = static_cast<uint8_t*>(c->v_exp);
  a.kx = static_cast<uint16_t*>(const_cast<void*>(K));
  a.vx = static_cast<uint16_t*>(const_cast<void*>(V));
  a.ks = k_stride;
  a.vs = v_stride;
  a.slots = slots;
  a.num_slots = c->pages * c->page_size;
  a.items = static_cast<uint32_t>(tokens * c->k_heads);
  a.div_heads = magic_encode(static_cast<uint32_t>(c->k_heads));
  a.div_page = magic_encode(static_cast<uint32_t>(c->page_size));
  a.heads = c->k_heads;
  a.page = c->page_size;
  const uint32_t groups = kCacheThreads / (c->head_dim / 8);
  const dim3 grid((a.items + groups - 1) / groups), block(kCacheThreads);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = dtype == GEMM_BF16;
  cudaError_t e;
  if constexpr (WRITE)
    e = c->head_dim == 128
            ? launch_pdl(bf16 ? cache_write_kernel<128, true> : cache_write_kernel<128, false>, grid, block, 0, s, a)
            : launch_pdl(bf16 ? cache_write_kernel<64, true> : cache_write_kernel<64, false>, grid, block, 0, s, a);
  else
    e = c->head_dim == 128
            ? launch_pdl(bf16 ? cache_read_kernel<128, true> : cache_read_kernel<128, false>, grid, block, 0, s, a)
            : launch_pdl(bf16 ? cache_read_kernel<64, true> : cache_read_kernel<64, false>, grid, block, 0, s, a);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_CUDA;
  }
  return GEMM_OK;
}

}  // namespace

bool cache_ok(const attn_cache_t& c) {
  return c.k && c.v && c.k_exp && c.v_exp && c.pages >= 1 && c.pages < (int64_t{1} << 31) && c.page_size >= 16 &&
         c.page_size <= 1024 && c.page_size % 16 == 0 && c.k_heads >= 1 && (c.head_dim == 64 || c.head_dim == 128);
}

}  // namespace lgt

extern "C" gemm_status_t attn_cache_write(const attn_cache_t* cache, const void* K, int64_t k_stride, const void* V,
                                          int64_t v_stride, const int32_t* slots, int64_t tokens, int32_t dtype,
                                          void* stream) {
  return lgt::run_cache<true>(cache, K, k_stride, V, v_stride, slots, tokens, dtype, stream);
}

extern "C" gemm_status_t attn_cache_read(const attn_cache_t* cache, const int32_t* slots, int64_t tokens, void* K,
                                         int64_t k_stride, void* V, int64_t v_stride, int32_t dtype, void* stream) {
  return lgt::run_cache<false>(cache, K, k_stride, V, v_stride, slots, tokens, dtype, stream);
}
