// matrix8.cuh -- what the kernels around the 8-bit matrices share: eight
// consecutive elements of a row in registers, their e4m3 codes, the place of
// a scale byte, and the dropout's random numbers.
//   matrix8.cu          -- values to codes and back
//   matrix8_multiply*.cu -- the products
//   rms_norm.cu         -- the norm and its backward pass
//   dropout.cu
#pragma once

#include <cuda_fp8.h>

#include "entry.h"
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

template <typename T>
__device__ __forceinline__ void load_eight(const T* p, float (&f)[8]);
template <>
__device__ __forceinline__ void load_eight<float>(const float* p, float (&f)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
template <>
__device__ __forceinline__ void load_eight<__nv_bfloat16>(const __nv_bfloat16* p, float (&f)[8]) {
  const uint4 r = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = __uint_as_float(w[k] << 16);
    f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}
template <>
__device__ __forceinline__ void load_eight<__half>(const __half* p, float (&f)[8]) {
  const uint4 r = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
    f[2 * k] = x.x;
    f[2 * k + 1] = x.y;
  }
}
template <typename T>
__device__ __forceinline__ void store_eight(T* p, const float (&f)[8]);
template <>
__device__ __forceinline__ void store_eight<float>(float* p, const float (&f)[8]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
}
template <>
__device__ __forceinline__ void store_eight<__nv_bfloat16>(__nv_bfloat16* p, const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 h = __float22bfloat162_rn(make_float2(f[2 * k], f[2 * k + 1]));
    w[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}
template <>
__device__ __forceinline__ void store_eight<__half>(__half* p, const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __half2 h = __float22half2_rn(make_float2(f[2 * k], f[2 * k + 1]));
    w[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
}

// The first n (0 to 8) elements at p, zeros after them: in one access where
// the rows allow it (vec) and all eight are there.
template <typename T>
__device__ __forceinline__ void load_some(const T* p, int n, bool vec, float (&f)[8]) {
  if (vec && n == 8) {
    load_eight<T>(p, f);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = j < n ? widen<T>(p[j]) : 0.f;
}
template <typename T>
__device__ __forceinline__ void store_some(T* p, int n, bool vec, const float (&f)[8]) {
  if (vec && n == 8) {
    store_eight<T>(p, f);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) p[j] = narrow<T>(f[j]);
}

// -------------------------------------------------------------------- codes --

// What values of a block with scale byte s are multiplied by before they are
// rounded to codes (0 where the block reads as NaN).
__device__ __forceinline__ float code_factor(uint32_t s) {
  return s == 255u ? 0.f : __uint_as_float((254u - s) << 23);
}
// Two codes, nearest even.  Where the block reads as NaN they are 0: a NaN or
// infinity times 0 is NaN, so that is asked for, not computed.
__device__ __forceinline__ uint32_t two_codes(float a, float b, float factor, bool nan) {
  if (nan) return 0u;
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(a, factor), __fmul_rn(b, factor)), __NV_SATFINITE,
                                            __NV_E4M3);
}
__device__ __forceinline__ uint32_t four_codes(const float* f, float factor, bool nan) {
  return two_codes(f[0], f[1], factor, nan) | two_codes(f[2], f[3], factor, nan) << 16;
}
// Eight codes' numbers before their block's unit.
__device__ __forceinline__ void widen_codes(uint2 c, float (&f)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t w = k < 2 ? c.x : c.y;
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((k & 1) ? w >> 16 : w & 0xFFFFu), __NV_E4M3);
    const float2 x = __half22float2(__half2(h));
    f[2 * k] = x.x;
    f[2 * k + 1] = x.y;
  }
}
// The bits of the largest magnitude of eight values (a NaN's are above all).
__device__ __forceinline__ uint32_t top_of(const float (&f)[8]) {
  uint32_t top = 0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(f[j]) & 0x7FFFFFFFu);
  return top;
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
// Drops among the eight elements from element i on.  A pair of elements (an
// even one and the next) has one hash; from an odd i the eight lie in five.
__device__ __forceinline__ void drop_eight(float (&f)[8], uint64_t i, const Drop& d, uint32_t key) {
  const uint64_t pair = i >> 1;
  const bool odd = i & 1;
  uint32_t h = hash_pair((uint32_t)pair * kHashPair + (uint32_t)(pair >> 32) * kHashHigh + key);
  if (odd) h >>= 16;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint64_t q = pair + k + 1;
    uint32_t next = 0u;
    if (k < 3 || odd) next = hash_pair((uint32_t)q * kHashPair + (uint32_t)(q >> 32) * kHashHigh + key);
    const uint32_t r0 = h & 0xFFFFu, r1 = odd ? next & 0xFFFFu : h >> 16;
    f[2 * k] = r0 < d.threshold ? 0.f : f[2 * k] * d.keep;
    f[2 * k + 1] = r1 < d.threshold ? 0.f : f[2 * k + 1] * d.keep;
    h = odd ? next >> 16 : next;
  }
}

}  // namespace dopt
