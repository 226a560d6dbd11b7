// matrix8.cuh -- what the kernels around the 8-bit matrices share: eight
// consecutive elements of a row in registers, their e4m3 codes, the place of
// a scale byte, and the dropout's random numbers.
//   matrix8.cu          -- values to codes and back
//   matrix8_multiply*.cu -- the products
//   rms_norm*.cu        -- the norm and its backward pass
//   dropout.cu
#pragma once

#include <cuda_fp8.h>

#include "entry.h"
#include "memset.h"
#include "tensors.cuh"

namespace dopt {

constexpr int kBlock8 = DOPT_MATRIX_BLOCK;

// Blocks of a row, and scale bytes of a matrix.
__host__ __device__ __forceinline__ int64_t row_blocks(int64_t cols) { return (cols + kBlock8 - 1) / kBlock8; }
__host__ __device__ __forceinline__ int64_t scale_groups(int64_t cols) { return (row_blocks(cols) + 3) / 4; }
__host__ __device__ __forceinline__ int64_t scale_size(int64_t rows, int64_t cols) {
  return (rows + 127) / 128 * scale_groups(cols) * 512;
}
// Place of the scale byte of row r, block b; groups = scale_groups(cols).
__device__ __forceinline__ int64_t scale_place(int64_t r, uint32_t b, uint32_t groups) {
  return ((r >> 7) * groups + (b >> 2)) * 512 + ((uint32_t)r & 31u) * 16u + (((uint32_t)r >> 5) & 3u) * 4u + (b & 3u);
}

// ------------------------------------------------- eight elements at a time --

// Whether rows of such elements can be read and written eight at a time.
inline bool eight_vectors(const void* p, int64_t ld, size_t elem) {
  return aligned_to(p, 16) && (ld * (int64_t)elem) % 16 == 0;
}

// Eight elements of a row as a load leaves them, widened only when they are
// used, so that a thread's loads are all under way before the first wait;
// then four pairs, for instructions on two fp32 numbers.
// VEC: consecutive elements in one streaming access (two for fp32); else every
// 32nd, so that a warp's accesses are consecutive, and not streaming: they
// share sectors with the next ones (509 bf16 columns to values 90 us against
// 81 so).
template <typename T, bool VEC>
struct Eight8 {
  T e[8];
  // of the elements at p, p + 32, ... those before `n`, zeros after them
  __device__ __forceinline__ void load(const T* p, int n) {
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = 32 * j < n ? p[32 * j] : narrow<T>(0.f);
  }
  __device__ __forceinline__ void widen8(float2 (&f)[4]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = make_float2(widen<T>(e[2 * k]), widen<T>(e[2 * k + 1]));
  }
  static __device__ __forceinline__ void store(T* p, int n, const float2 (&f)[4]) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (32 * j < n) p[32 * j] = narrow<T>(j & 1 ? f[j / 2].y : f[j / 2].x);
  }
};
template <>
struct Eight8<float, true> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p, int n) {
    a = b = make_float4(0.f, 0.f, 0.f, 0.f);
    if (n > 0) {
      a = __ldcs(reinterpret_cast<const float4*>(p));
      b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    }
  }
  __device__ __forceinline__ void widen8(float2 (&f)[4]) const {
    f[0] = make_float2(a.x, a.y), f[1] = make_float2(a.z, a.w), f[2] = make_float2(b.x, b.y), f[3] = make_float2(b.z, b.w);
  }
  static __device__ __forceinline__ void store(float* p, int n, const float2 (&f)[4]) {
    if (n <= 0) return;
    __stcs(reinterpret_cast<float4*>(p), make_float4(f[0].x, f[0].y, f[1].x, f[1].y));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(f[2].x, f[2].y, f[3].x, f[3].y));
  }
};
// Two 16-bit elements of a word.
template <typename T>
__device__ __forceinline__ float2 widen_pair(uint32_t w);
template <>
__device__ __forceinline__ float2 widen_pair<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 widen_pair<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t narrow_pair(float2 x);
template <>
__device__ __forceinline__ uint32_t narrow_pair<__nv_bfloat16>(float2 x) {
  const __nv_bfloat162 h = __float22bfloat162_rn(x);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t narrow_pair<__half>(float2 x) {
  const __half2 h = __float22half2_rn(x);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
struct Eight8<T, true> {
  uint4 r;
  __device__ __forceinline__ void load(const T* p, int n) {
    r = make_uint4(0u, 0u, 0u, 0u);
    if (n > 0) r = __ldcs(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void widen8(float2 (&f)[4]) const {
    f[0] = widen_pair<T>(r.x), f[1] = widen_pair<T>(r.y), f[2] = widen_pair<T>(r.z), f[3] = widen_pair<T>(r.w);
  }
  static __device__ __forceinline__ void store(T* p, int n, const float2 (&f)[4]) {
    if (n <= 0) return;
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(narrow_pair<T>(f[0]), narrow_pair<T>(f[1]), narrow_pair<T>(f[2]), narrow_pair<T>(f[3])));
  }
};
// f rounded to T and widened again.
template <typename T>
__device__ __forceinline__ void round_eight(float2 (&f)[4]) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = widen_pair<T>(narrow_pair<T>(f[k]));
  }
}
__device__ __forceinline__ float2 both_of(float x) { return make_float2(x, x); }

// -------------------------------------------------------------------- codes --

// What values of a block are multiplied by before they are rounded to codes,
// 2^(127 - s) as (254 - s) << 23, straight from the bits of the block's
// largest magnitude; its scale byte, and whether all of it reads as NaN.
struct BlockScale {
  uint32_t factor;
  bool nan;
  __device__ __forceinline__ explicit BlockScale(uint32_t top) {
    const uint32_t e = (top + 0x1FFFFFu) & 0xFF800000u;  // m_scale_of's exponent, in place
    nan = e >= 255u << 23;
    factor = min((262u << 23) - e, 246u << 23);
  }
  __device__ __forceinline__ float2 up() const {
    const float f = __uint_as_float(factor);
    return make_float2(f, f);
  }
  __device__ __forceinline__ uint32_t byte() const { return nan ? 255u : 254u - (factor >> 23); }
};
// Codes of four values, nearest even, before the question whether the block
// reads as NaN (all its codes are 0 then, whatever the conversion gave).
__device__ __forceinline__ uint32_t four_codes(float2 a, float2 b, float2 up) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(__fmul2_rn(a, up), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(__fmul2_rn(b, up), __NV_SATFINITE, __NV_E4M3);
  return __byte_perm(lo, hi, 0x5410);
}
__device__ __forceinline__ uint32_t four_codes(float2 a, float2 b, const BlockScale& s) {
  const uint32_t c = four_codes(a, b, s.up());
  return s.nan ? 0u : c;
}
// Eight codes' numbers before their block's unit.
__device__ __forceinline__ void widen_codes(uint2 c, float2 (&f)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t w = k < 2 ? c.x : c.y;
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((k & 1) ? w >> 16 : w & 0xFFFFu), __NV_E4M3);
    f[k] = __half22float2(__half2(h));
  }
}
// The bits of the larger magnitude of two values and `top` (a NaN's are above
// all).
__device__ __forceinline__ uint32_t top_of(uint32_t top, float2 f) {
  return __vimax3_u32(top, __float_as_uint(f.x) & 0x7FFFFFFFu, __float_as_uint(f.y) & 0x7FFFFFFFu);
}

// ------------------------------------------------------------------ dropout --

// A call's dropout: threshold 0 where it has none.
struct Drop {
  const int64_t* d_step;
  uint32_t threshold;
  uint32_t key;  // seed, site and the host's step
  float keep;    // 65536 / (65536 - threshold)
};
inline Drop make_drop(const dopt_drop& d, uint32_t threshold) {
  return Drop{d.d_step, threshold, d.seed + d.site * kHashTensor + (uint32_t)d.step * kHashStep,
              (float)(65536.0 / (65536.0 - threshold))};
}
constexpr uint32_t kHashHigh = 0x3C6EF372u;
__device__ __forceinline__ uint32_t drop_key(const Drop& d) {
  return d.key + (d.threshold && d.d_step ? (uint32_t)*d.d_step * kHashStep : 0u);
}
__device__ __forceinline__ uint32_t drop_hash(uint64_t pair, uint32_t key) {
  return hash_pair((uint32_t)pair * kHashPair + (uint32_t)(pair >> 32) * kHashHigh + key);
}
// Drops among eight elements from element i on: consecutive ones with i a
// multiple of 8 (VEC), two to a hash; or every 32nd.
template <bool VEC>
__device__ __forceinline__ void drop_eight(float2 (&f)[4], uint64_t i, const Drop& d, uint32_t key) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t r0, r1;
    if constexpr (VEC) {
      const uint32_t h = drop_hash((i >> 1) + k, key);
      r0 = h & 0xFFFFu;
      r1 = h >> 16;
    } else {
      const uint64_t at = i + 64 * k;  // i + 64 k and i + 64 k + 32 have one parity
      const uint32_t h0 = drop_hash(at >> 1, key), h1 = drop_hash((at + 32) >> 1, key);
      r0 = at & 1 ? h0 >> 16 : h0 & 0xFFFFu;
      r1 = at & 1 ? h1 >> 16 : h1 & 0xFFFFu;
    }
    const float2 kept = __fmul2_rn(f[k], both_of(d.keep));
    f[k] = make_float2(r0 < d.threshold ? 0.f : kept.x, r1 < d.threshold ? 0.f : kept.y);
  }
}

}  // namespace dopt
