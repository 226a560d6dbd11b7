// tensors_adamw8.cu -- AdamW over a list of tensors with the moments in 8
// bits, and the moments' conversion between values and 8-bit codes.
//
// The update reads grad, weight and both codes of every element once and
// writes weight, 16-bit param and both codes once: 16 bytes per element with
// bf16 or fp16 grads and params, or with both in fp32 (and 4 scale bytes per
// block).  Against 28 to 30 bytes with fp32 moments that leaves the same
// arithmetic and the encoding half the time, about 90 issue slots per element
// at the memory's rate, so both count: the moments' arithmetic runs two
// elements per instruction, codes are made two at a time, and the inputs
// come through a ring in shared memory.  A warp has a block of 256 elements
// at a time, so a block's largest moments are one warp reduction each.
// Measured on 1.35e9 bf16 elements: 3.14 ms, 6.9 TB/s (1.02 of the copy
// bandwidth); as many fp32 params and grads: 3.06 ms, 7.05 TB/s.
#include <cuda_fp8.h>

#include "tensors.cuh"

namespace dopt {

// Three CTAs per SM and three slots per warp: 20 KB per slot and CTA, 180 KB of
// the SM's shared memory.  Four CTAs (64 registers) were 7 % slower, two slots
// 5 %; four slots leave room for two CTAs only (21 % slower).
// Rounds of a CTA's walk over the tiles (see launch_walk): the best of 1 to 64
// and of no limit, which took 3490 us on 1.35e9 bf16 elements against 3133.
constexpr int kRing8 = 3, kCtas8 = 3, kRounds8 = 24;
static_assert(kMomentBlock == 256 && kAdamTile % kMomentBlock == 0, "one warp per block, 8 elements per lane");

__device__ __forceinline__ uint32_t exponent_of(uint32_t bits, uint32_t up) { return (bits + up) >> 23; }

__device__ __forceinline__ float m_unit(uint32_t s) {
  return s == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(s << 23);
}
__device__ __forceinline__ uint32_t hash_pair(uint32_t x) {
  uint64_t q = (uint64_t)x * kHashMul1;
  x = (uint32_t)q ^ (uint32_t)(q >> 32);
  q = (uint64_t)x * kHashMul2;
  return (uint32_t)q ^ (uint32_t)(q >> 32);
}

// A block's scales from the bits of its largest magnitude: 255 where that is
// not finite or above the largest code.
__device__ __forceinline__ uint32_t m_scale_of(uint32_t top) {
  const uint32_t e = exponent_of(top, 0x1FFFFFu);
  return e >= 255u ? 255u : max((int)e - 8, 8);
}
__device__ __forceinline__ uint32_t v_scale_of(uint32_t top) {
  const uint32_t e = exponent_of(top, 0x0FFFFFu);
  return e >= 255u ? 255u : (uint32_t)max((int)e - 31, 0);
}
// Eight consecutive fp32 elements in one 32-byte access (streaming: read
// once, written once).
__device__ __forceinline__ void load8(const float* p, float2* x) {
  asm volatile("ld.global.cs.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(x[0].x), "=f"(x[0].y), "=f"(x[1].x), "=f"(x[1].y), "=f"(x[2].x), "=f"(x[2].y), "=f"(x[3].x), "=f"(x[3].y)
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void store8(float* p, const float2* x) {
  asm volatile("st.global.cs.v8.f32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"f"(x[0].x), "f"(x[0].y), "f"(x[1].x),
               "f"(x[1].y), "f"(x[2].x), "f"(x[2].y), "f"(x[3].x), "f"(x[3].y), "l"(p)
               : "memory");
}

// Eight consecutive elements of a type as four pairs: what a load leaves in
// registers until it is widened, and the store.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  struct Raw {
    float2 x[4];
  };
  static __device__ __forceinline__ void load(const float* p, Raw& r) { load8(p, r.x); }
  static __device__ __forceinline__ void widen8(const Raw& r, float2* x) {
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = r.x[k];
  }
  static __device__ __forceinline__ void store(float* p, const float2* x) { store8(p, x); }
};
template <>
struct Eight<__nv_bfloat16> {
  using Raw = uint4;
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, Raw& r) { r = __ldcs(reinterpret_cast<const uint4*>(p)); }
  static __device__ __forceinline__ void widen8(const Raw& r, float2* x) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float2* x) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 h = __float22bfloat162_rn(x[k]);
      w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  }
};
template <>
struct Eight<__half> {
  using Raw = uint4;
  static __device__ __forceinline__ void widen8(const Raw& r, float2* x) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
  }
  static __device__ __forceinline__ void store(__half* p, const float2* x) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __half2 h = __float22half2_rn(x[k]);
      w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  }
};

// Element j of four pairs.
__device__ __forceinline__ float& elem(float2* x, int j) { return j & 1 ? x[j / 2].y : x[j / 2].x; }

// exp_avg codes (two words, eight codes) as the numbers they are before
// their block's unit.
__device__ __forceinline__ void widen_m(uint2 mc, float2* m) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t w = k < 2 ? mc.x : mc.y;
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((k & 1) ? w >> 16 : w & 0xFFFFu), __NV_E4M3);
    m[k] = __half22float2(__half2(h));
  }
}
// exp_avg_sq codes as values: base + the code at bits 20..27, and 0 for
// code 0 (checked for all eight at once; rare but for blocks never touched).
__device__ __forceinline__ void widen_v(uint2 vc, uint32_t s, float2* v) {
  const uint32_t base = s << 23;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    elem(v, j) = __uint_as_float(__byte_perm(j < 4 ? vc.x : vc.y, 0, 0x4440 + (j & 3)) * 0x100000u + base);
  const uint32_t zero = ((vc.x - 0x01010101u) & ~vc.x) | ((vc.y - 0x01010101u) & ~vc.y);
  if ((zero & 0x80808080u) || s == 255u) {  // a byte is 0 (or, harmlessly, 1 above a 0)
    const float none = s == 255u ? __uint_as_float(0x7FC00000u) : 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (s == 255u || !(((j < 4 ? vc.x : vc.y) >> (8 * (j & 3))) & 0xFFu)) elem(v, j) = none;
  }
}

// Largest of three magnitudes, NaN above all.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// The largest magnitude of the warp's elements, eight per lane, as fp32 bits
// (their order is that of the magnitudes, NaN above all).
__device__ __forceinline__ uint32_t block_top(const float2* x) {
  float t = max3_abs(x[0].x, x[0].y, x[1].x);
  t = max3_abs(t, x[1].y, x[2].x);
  t = max3_abs(t, x[2].y, x[3].x);
  t = max3_abs(t, x[3].y, x[3].y);
  return __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(t));
}

__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// The least of eight that are not NaN.
__device__ __forceinline__ float least_of(const float2* x) {
  return min3(min3(min3(x[0].x, x[0].y, x[1].x), x[1].y, x[2].x), min3(x[2].y, x[3].x, x[3].y), x[3].y);
}

__device__ __forceinline__ uint2 narrow_m(const float2* m, uint32_t s) {
  const float up = __uint_as_float((254u - s) << 23);
  const float2 up2 = make_float2(up, up);
  uint32_t h[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) h[k] = __nv_cvt_float2_to_fp8x2(__fmul2_rn(m[k], up2), __NV_SATFINITE, __NV_E4M3);
  return s == 255u ? make_uint2(0u, 0u) : make_uint2(__byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410));
}
// r16: the elements' rounding bits, two per word (0x8000: nearest); least: of
// the elements.  Two codes
// at a time in the halves of a word: the fp32 patterns' upper halves, held
// at the smallest code or above, less the base, shifted down to bytes.  The
// scale keeps codes at most 255.
__device__ __forceinline__ uint2 narrow_v(const float2* v, uint32_t s, const uint32_t* r16, float least) {
  const uint32_t base16 = s * 0x00800080u, least16 = base16 + 0x00100010u;
  uint32_t h[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t a = __float_as_uint(v[k].x) + ((r16[k] & 0xFFFFu) << 4);
    const uint32_t b = __float_as_uint(v[k].y) + ((r16[k] >> 16) << 4);
    h[k] = (__vmaxu2(__byte_perm(a, b, 0x7632), least16) - base16) >> 4;  // codes in bytes 0 and 2
  }
  uint2 c = make_uint2(__byte_perm(h[0], h[1], 0x6420), __byte_perm(h[2], h[3], 0x6420));
  if (least == 0.f) {  // zeros have code 0
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if ((j & 1 ? v[j / 2].y : v[j / 2].x) == 0.f) (j < 4 ? c.x : c.y) &= ~(0xFFu << (8 * (j & 3)));
    }
  }
  return s == 255u ? make_uint2(0u, 0u) : c;
}

// AdamW on eight elements, in fp32, two per instruction but for the moments'
// sums: the moments round each operation once, bit for bit as the fp32 ones
// do, and a packed sum of packed products would be compiled into a fused
// multiply-add whatever its rounding mode says (found by comparing results
// on sm_103a; 2 % of the instructions).  The weight's update takes the
// hardware's approximate root and reciprocal, each within 2^-22 of the exact.
// Correctly rounded ones cost half of the kernel's instructions, which then
// bound it: 5.0 ms against 3.8 on 1.35e9 elements.  The root takes subnormals
// for 0, and eps may be smaller than theirs (1.1e-19 at 2^-126), so a lane
// that has such a v (or a zero) takes those roots again, of v 2^24 times as
// large (0.1 to 0.5 %; a root that keeps subnormals in every lane costs 0.7 to
// 1.5 %, and 11 % on tensors off the vector grid).
struct Adam8 {
  float2 inv_scale, c, decay, b1, b2, omb1, omb2, minus_size, inv_bc2, eps;
};
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float root(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 sum2(float2 a, float2 b) {
  return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}
// m arrives without its block's unit, which b1 carries (a power of two: the
// product is the same, unless b1 times the unit is subnormal, which takes a b1
// below 2^-7: at most 2^-141 off, where codes are 2^-128 apart or more.
// Multiplying m by the unit first instead, under a branch on b1, costs 0.3 %,
// and 7 % off the vector grid).  Returns the least v.
__device__ __forceinline__ float adamw_pairs(const Adam8& a, float2 b1_unit, float2* g, float2* w, float2* m, float2* v) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 gk = __fmul2_rn(__fmul2_rn(g[k], a.inv_scale), a.c);
    m[k] = sum2(__fmul2_rn(b1_unit, m[k]), __fmul2_rn(a.omb1, gk));
    v[k] = sum2(__fmul2_rn(a.b2, v[k]), __fmul2_rn(__fmul2_rn(a.omb2, gk), gk));
  }
  float2 r[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) r[k] = make_float2(root(v[k].x), root(v[k].y));
  const float least = least_of(v);
  if (least < 0x1p-126f) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (elem(v, j) < 0x1p-126f) elem(r, j) = __fmul_rn(root(__fmul_rn(elem(v, j), 0x1p24f)), 0x1p-12f);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 denom = __ffma2_rn(r[k], a.inv_bc2, a.eps);
    const float2 u = __fmul2_rn(m[k], make_float2(reciprocal(denom.x), reciprocal(denom.y)));
    w[k] = __ffma2_rn(a.minus_size, u, __fmul2_rn(w[k], a.decay));
  }
  return least;
}

// Where a tile lies.  All of it is the same for the whole CTA, so that
// addresses are a uniform base plus a thread's constant offset.
struct Place8 {
  int si;         // the tensor
  int64_t first;  // the tile's first element
  int n;          // elements of the tensor from there, at most kAdamTile
};
template <typename P>
__device__ __forceinline__ Place8 place_tile(const P& p, int t, int si) {
  const AdamSeg& sg = p.seg[si];
  Place8 a;
  a.si = si;
  a.first = (int64_t)(t - sg.tile0) * kAdamTile;
  a.n = (int)min((int64_t)kAdamTile, sg.len - a.first);
  if (!DOPT_TILE_OK(p, kSiteListAdam8, a.first, a.n, sg.len)) a.n = 0;
  return a;
}

template <typename T>
__device__ __forceinline__ T* at_offset(T* base, uint32_t elems) {
  return reinterpret_cast<T*>(reinterpret_cast<char*>(base) + elems * (uint32_t)sizeof(T));
}
template <typename T>
__device__ __forceinline__ const T* at_offset(const T* base, uint32_t elems) {
  return reinterpret_cast<const T*>(reinterpret_cast<const char*>(base) + elems * (uint32_t)sizeof(T));
}

// A whole block's inputs reach its warp through a ring of kRing8 slots of
// shared memory per warp, filled by asynchronous copies kRing8 - 1 tiles
// ahead: the loads in flight then depend neither on registers nor on the
// number of resident warps, both of which the update's arithmetic limits.
// Each lane copies 16-byte pieces (grads, weights, then exp_avg's and
// exp_avg_sq's codes); each warp waits for its own copies only.
struct Ring8 {
  static constexpr int kGrad = kMomentBlock * 4, kWeight = kMomentBlock * 4, kCodes = kMomentBlock;  // parts' bytes
  static constexpr int kSlot = kGrad + kWeight + 2 * kCodes;
  static constexpr size_t kBytes = (size_t)kRing8 * (kThreads / 32) * kSlot;
};
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Where 16-byte piece c of an fp32 array lies in its part of a slot: pieces 2i
// and 2i + 1 are lane i's, and the swap of every second group of eight lets
// eight lanes read theirs from eight different bank groups.
__device__ __forceinline__ uint32_t piece_at(uint32_t c) { return (c ^ ((c >> 3) & 1u)) * 16u; }

// Whether a warp's block comes through the ring: it is whole, and the
// tensor's arrays start on 16-byte boundaries.
__device__ __forceinline__ bool through_ring(const AdamSeg& sg, const Place8& a) {
  return sg.shift == 0 && (int)(threadIdx.x / 32 + 1) * kMomentBlock <= a.n;
}
template <typename P>
__device__ __forceinline__ void fetch_block(const P& p, const Place8& a, uint32_t slot, uint32_t& scales) {
  const AdamSeg& sg = p.seg[a.si];
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if ((int)(warp * kMomentBlock) < a.n)
    scales = *at_offset(sg.m_scale + a.first / kMomentBlock, warp) |
             ((uint32_t)*at_offset(sg.v_scale + a.first / kMomentBlock, warp) << 8);
  if (!through_ring(sg, a)) return;
  const char* w = reinterpret_cast<const char*>(sg.weight + a.first);
  if (sg.grad_dtype == DOPT_F32) {
    const char* g = reinterpret_cast<const char*>(static_cast<const float*>(sg.grad) + a.first);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t c = k * 32 + lane;
      copy16(slot + piece_at(c), g + warp * Ring8::kGrad + c * 16u);
    }
  } else {
    const char* g = reinterpret_cast<const char*>(static_cast<const uint16_t*>(sg.grad) + a.first);
    copy16(slot + lane * 16u, g + warp * (kMomentBlock * 2) + lane * 16u);
  }
  slot += Ring8::kGrad;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t c = k * 32 + lane;
    copy16(slot + piece_at(c), w + warp * Ring8::kWeight + c * 16u);
  }
  slot += Ring8::kWeight;
  const uint8_t* codes = static_cast<const uint8_t*>(lane < 16 ? sg.m : sg.v) + a.first;
  copy16(slot + lane * 16u, codes + warp * kMomentBlock + (lane & 15u) * 16u);
}

__device__ __forceinline__ uint4 shared16(uint32_t at) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(at) : "memory");
  return r;
}
__device__ __forceinline__ uint2 shared8(uint32_t at) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(at) : "memory");
  return r;
}
__device__ __forceinline__ void shared_floats(uint32_t at, uint32_t lane, float2* x) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint4 r = shared16(at + piece_at(2 * lane + k));
    x[2 * k] = make_float2(__uint_as_float(r.x), __uint_as_float(r.y));
    x[2 * k + 1] = make_float2(__uint_as_float(r.z), __uint_as_float(r.w));
  }
}
// A lane's eight elements of its warp's slot.
template <typename GT>
__device__ __forceinline__ void from_ring(uint32_t slot, uint32_t lane, float2* g, float2* w, uint2& mc, uint2& vc) {
  if constexpr (sizeof(GT) == 4)
    shared_floats(slot, lane, g);
  else
    Eight<GT>::widen8(shared16(slot + lane * 16u), g);
  shared_floats(slot + Ring8::kGrad, lane, w);
  mc = shared8(slot + Ring8::kGrad + Ring8::kWeight + lane * 8u);
  vc = shared8(slot + Ring8::kGrad + Ring8::kWeight + Ring8::kCodes + lane * 8u);
}

// Updates a warp's block that came through the ring.  key: the hash's
// argument for the tile's first pair.
template <typename PT, typename GT>
__device__ __forceinline__ void step_block(const AdamSeg& sg, const Place8& a, uint32_t slot, uint32_t scales,
                                           const Adam8& ad, uint32_t key) {
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, at = threadIdx.x * 8;
  float2 g[4], w[4], m[4], v[4];
  uint2 mc, vc;
  from_ring<GT>(slot, lane, g, w, mc, vc);
  widen_m(mc, m);
  widen_v(vc, scales >> 8, v);
  const float least = adamw_pairs(ad, both(__fmul_rn(ad.b1.x, m_unit(scales & 0xFFu))), g, w, m, v);
  store8(at_offset(sg.weight + a.first, at), w);
  if constexpr (sizeof(PT) == 2) Eight<PT>::store(at_offset(static_cast<PT*>(sg.param) + a.first, at), w);
  const uint32_t ms = m_scale_of(block_top(m)), vs = v_scale_of(block_top(v));
  uint32_t r16[4];
  const uint32_t y = key + (at >> 1) * kHashPair;
#pragma unroll
  for (int k = 0; k < 4; ++k) r16[k] = hash_pair(y + k * kHashPair);
  if (lane == 0) {
    *at_offset(sg.m_scale + a.first / kMomentBlock, warp) = (uint8_t)ms;
    *at_offset(sg.v_scale + a.first / kMomentBlock, warp) = (uint8_t)vs;
  }
  __stcs(reinterpret_cast<uint2*>(at_offset(static_cast<uint8_t*>(sg.m) + a.first, at)), narrow_m(m, ms));
  __stcs(reinterpret_cast<uint2*>(at_offset(static_cast<uint8_t*>(sg.v) + a.first, at)), narrow_v(v, vs, r16, least));
}

// Updates a block of n elements from element `first` of a tensor (its ragged
// last one, or any where the arrays have no common vector boundary).  Element
// j of a lane is 32 apart from the next: consecutive lanes, consecutive
// elements.  One body for every type: five copies of it beside the path above
// cost that path 3 %, and a call out of line half its speed (its arguments go
// through memory).
__device__ __forceinline__ void step_loose(const AdamSeg& sg, int64_t first, int n, uint32_t scales, const Adam8& ad, uint32_t key) {
  const uint32_t lane = threadIdx.x % 32;
  float* const wp = sg.weight + first + lane;
  uint8_t* const mp = static_cast<uint8_t*>(sg.m) + first + lane;
  uint8_t* const vp = static_cast<uint8_t*>(sg.v) + first + lane;
  float2 g[4], w[4], m[4], v[4];
  uint32_t mw[2] = {0u, 0u}, vw[2] = {0u, 0u};
  // every load before any use of one: the path has no copies ahead
  if (sg.grad_dtype == DOPT_F32) {
    const float* const gp = static_cast<const float*>(sg.grad) + first + lane;
#pragma unroll
    for (int j = 0; j < 8; ++j) elem(g, j) = (int)lane + j * 32 < n ? gp[j * 32] : 0.f;
  } else {
    const uint16_t* const gp = static_cast<const uint16_t*>(sg.grad) + first + lane;
    uint16_t r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = (int)lane + j * 32 < n ? gp[j * 32] : 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      elem(g, j) = sg.grad_dtype == DOPT_BF16 ? __uint_as_float((uint32_t)r[j] << 16) : __half2float(__ushort_as_half(r[j]));
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const bool in = (int)lane + j * 32 < n;
    elem(w, j) = in ? wp[j * 32] : 0.f;
    mw[j / 4] |= (in ? (uint32_t)mp[j * 32] : 0u) << (8 * (j & 3));
    vw[j / 4] |= (in ? (uint32_t)vp[j * 32] : 0u) << (8 * (j & 3));
  }
  widen_m(make_uint2(mw[0], mw[1]), m);
  widen_v(make_uint2(vw[0], vw[1]), scales >> 8, v);
  const float least = adamw_pairs(ad, both(__fmul_rn(ad.b1.x, m_unit(scales & 0xFFu))), g, w, m, v);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if ((int)lane + j * 32 < n) {
      wp[j * 32] = elem(w, j);
      store_param(sg.param, first + lane + j * 32, sg.param_dtype, elem(w, j));
    } else {
      elem(m, j) = elem(v, j) = 0.f;  // past the end: no part in the scales (NaN blocks)
    }
  }
  const uint32_t ms = m_scale_of(block_top(m)), vs = v_scale_of(block_top(v));
  uint32_t r16[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t y = key + ((uint32_t)(first >> 1) + (lane >> 1) + k * 32) * kHashPair;
    r16[k] = __byte_perm(hash_pair(y), hash_pair(y + 16 * kHashPair), (lane & 1) ? 0x7632 : 0x5410);
  }
  const uint2 mc = narrow_m(m, ms), vc = narrow_v(v, vs, r16, least);
  if (lane == 0) {
    sg.m_scale[first / kMomentBlock] = (uint8_t)ms;
    sg.v_scale[first / kMomentBlock] = (uint8_t)vs;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if ((int)lane + j * 32 < n) {
      mp[j * 32] = (uint8_t)((j < 4 ? mc.x : mc.y) >> (8 * (j & 3)));
      vp[j * 32] = (uint8_t)((j < 4 ? vc.x : vc.y) >> (8 * (j & 3)));
    }
  }
}

// The block's update for its tensor's types (the same for the whole CTA).
// key: the hash's argument for the tensor's first pair.
__device__ __forceinline__ void step_block_of(const AdamSeg& sg, const Place8& a, uint32_t slot, uint32_t scales,
                                              const Adam8& ad, uint32_t key) {
  if (!through_ring(sg, a)) {
    const int64_t block = (int64_t)(threadIdx.x / 32) * kMomentBlock;
    step_loose(sg, a.first + block, min(a.n - (int)block, kMomentBlock), scales, ad, key);
    return;
  }
  key += (uint32_t)(a.first >> 1) * kHashPair;
  if (sg.param_dtype == DOPT_BF16) {
    if (sg.grad_dtype == DOPT_BF16)
      step_block<__nv_bfloat16, __nv_bfloat16>(sg, a, slot, scales, ad, key);
    else
      step_block<__nv_bfloat16, float>(sg, a, slot, scales, ad, key);
  } else if (sg.param_dtype == DOPT_F16) {
    if (sg.grad_dtype == DOPT_F16)
      step_block<__half, __half>(sg, a, slot, scales, ad, key);
    else
      step_block<__half, float>(sg, a, slot, scales, ad, key);
  } else {
    step_block<float, float>(sg, a, slot, scales, ad, key);
  }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, kCtas8) tensors_adamw8(const __grid_constant__ AdamParamsT<CAP> p) {
  extern __shared__ uint4 ring[];
  uint32_t slot0;
  asm("{.reg .u64 t; cvta.to.shared.u64 t, %1; cvt.u32.u64 %0, t;}" : "=r"(slot0) : "l"(ring));
  slot0 += threadIdx.x / 32 * (kRing8 * Ring8::kSlot);
  const TileWalk walk = tile_walk(p);
  int t = walk.first;
  Place8 cur = {}, ahead;
  uint32_t scales[kRing8];  // of the tiles in flight, this one's first
  int tensor[kRing8];
  int hop = 1;
  if (!p.early) wait_for_prior_grids();
  // the first kRing8 - 1 tiles; the launch before this one, when it is of
  // the same call, writes none of what they read
  if (t < walk.end) cur = place_tile(p, t, find_seg(p, t));
  ahead = cur;
  int ta = t;
#pragma unroll
  for (int k = 0; k < kRing8 - 1; ++k) {
    if (ta < walk.end) {
      if (k) ahead = place_tile(p, ta, next_seg(p, ahead.si, ta, hop));
      tensor[k] = ahead.si;
      fetch_block(p, ahead, slot0 + k * Ring8::kSlot, scales[k]);
      ta += p.stride;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  if (p.early) wait_for_prior_grids();
  if (t >= walk.end || (p.found_inf && *p.found_inf)) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  Adam8 ad;
  ad.inv_scale = both(p.inv_scale);
  ad.c = both(p.coef ? *p.coef : 1.f);
  ad.b1 = both(p.b1);
  ad.b2 = both(p.b2);
  ad.omb1 = both(p.omb1);
  ad.omb2 = both(p.omb2);
  // The reciprocal takes subnormals for 0, so a denominator near them is formed
  // 2^24 times as large, as is the step size; 2^-126 there keeps an eps that
  // is 0 in fp32 from dividing 0 by 0.
  const float lift = p.eps < 0x1p-100f ? 0x1p24f : 1.f;
  ad.minus_size = both(-lift * (p.dev ? p.dev->step_size : p.step_size));
  ad.inv_bc2 = both(lift * __fdiv_rn(1.f, p.dev ? p.dev->bc2_sqrt : p.bc2_sqrt));
  ad.eps = both(fmaxf(lift * p.eps, 0x1p-126f));
  ad.decay = both(decay_of_seg(p, p.seg[cur.si]));
  const uint32_t key = p.key + (p.d_step ? (uint32_t)*p.d_step * kHashStep : 0u);
  uint32_t slot = slot0, slot_ahead = slot0 + (kRing8 - 1) * Ring8::kSlot;
  const uint32_t slot_end = slot0 + kRing8 * Ring8::kSlot;
  for (;;) {
    if (ta < walk.end) {
      ahead = place_tile(p, ta, next_seg(p, ahead.si, ta, hop));
      tensor[kRing8 - 1] = ahead.si;
      fetch_block(p, ahead, slot_ahead, scales[kRing8 - 1]);
      ta += p.stride;
    }
    asm volatile("cp.async.commit_group;\n cp.async.wait_group %0;" ::"n"(kRing8 - 1) : "memory");
    __syncwarp();  // the warp's copies, not this lane's alone
    if ((int)(threadIdx.x / 32 * kMomentBlock) < cur.n)
      step_block_of(p.seg[cur.si], cur, slot, scales[0], ad, key + p.seg[cur.si].key);
    t += p.stride;
    if (t >= walk.end) break;
    const Place8 next = place_tile(p, t, tensor[1]);
    if (next.si != cur.si) ad.decay = both(decay_of_seg(p, p.seg[next.si]));
    cur = next;
#pragma unroll
    for (int k = 0; k + 1 < kRing8; ++k) {
      scales[k] = scales[k + 1];
      tensor[k] = tensor[k + 1];
    }
    slot_ahead = slot;
    slot = slot + Ring8::kSlot == slot_end ? slot0 : slot + Ring8::kSlot;
    __syncwarp();  // every lane has read the slot before it is filled again
  }
}

int launch_tensors_adamw8(AdamParamsT<kAdamCap>& p, cudaStream_t s) {
  const char* what = "tensors_adamw8 launch";
  if (p.n_seg <= kAdamSmallCap) {
    AdamParamsT<kAdamSmallCap> small = compact_table<AdamParamsT<kAdamSmallCap>, AdamHead>(p);
    return launch_walk<tensors_adamw8<kAdamSmallCap>, Ring8::kBytes, kRounds8>(small, s, what, true);
  }
  return launch_walk<tensors_adamw8<kAdamCap>, Ring8::kBytes, kRounds8>(p, s, what, true);
}

// ------------------------------------------------------- pack and unpack --

// Packing takes one warp per block, eight elements per lane: consecutive ones
// in vectors where every array has its first element on a vector boundary and
// the block is whole, else 32 apart.  A thread loads its next tile's values
// before it packs this one's when they are bf16: 1.3e8 elements take 150 us
// so and 162 without; fp32 ones 190 us without, at the copy bandwidth, and
// 199 with.  Five CTAs per SM; six spill (fp32 206 us).  16 rounds of a walk:
// 1.35e9 fp32 elements 1841 us, 7.31 TB/s, against 1915 without a limit.
template <typename VT>
constexpr bool kPackAhead = sizeof(VT) == 2;
constexpr int kPackCtas = 5, kPackRounds = 16;
template <typename VT>
struct Values8 {
  typename Eight<VT>::Raw m, v;
};
template <typename P>
__device__ __forceinline__ Place8 place_values(const P& p, int t, int si) {
  const MomentSeg& sg = p.seg[si];
  Place8 a;
  a.si = si;
  a.first = (int64_t)(t - sg.tile0) * kAdamTile;
  a.n = (int)min((int64_t)kAdamTile, sg.len - a.first);
  if (!DOPT_TILE_OK(p, kSiteListMoments, a.first, a.n, sg.len)) a.n = 0;
  return a;
}
__device__ __forceinline__ bool whole_block(const MomentSeg& sg, const Place8& a) {
  return sg.vec && (int)(threadIdx.x / 32 + 1) * kMomentBlock <= a.n;
}
template <typename VT, typename P>
__device__ __forceinline__ void load_values(const P& p, const Place8& a, Values8<VT>& x) {
  const MomentSeg& sg = p.seg[a.si];
  if (!whole_block(sg, a)) return;
  if (sg.m) Eight<VT>::load(at_offset(static_cast<const VT*>(sg.m) + a.first, threadIdx.x * 8), x.m);
  if (sg.v) Eight<VT>::load(at_offset(static_cast<const VT*>(sg.v) + a.first, threadIdx.x * 8), x.v);
}
// Codes and scale of one moment's values of a warp's block.
__device__ __forceinline__ uint2 pack_m_values(const float2* m, uint32_t& s) {
  s = m_scale_of(block_top(m));
  return narrow_m(m, s);
}
__device__ __forceinline__ uint2 pack_v_values(float2* v, uint32_t& s) {
  // -0 is 0; what is below 0 is not a second moment: its sign bit puts it
  // above every finite value here, so its block becomes NaN
  uint32_t top = 0u;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[k] = __fadd2_rn(v[k], make_float2(0.f, 0.f));
    top = __vimax3_u32(top, __float_as_uint(v[k].x), __float_as_uint(v[k].y));
  }
  s = v_scale_of(min(__reduce_max_sync(0xFFFFFFFFu, top), 0x7FFFFFFFu));
  const uint32_t nearest[4] = {0x80008000u, 0x80008000u, 0x80008000u, 0x80008000u};
  return narrow_v(v, s, nearest, least_of(v));
}

// A lane's elements of a block that is not read in vectors, and its codes'
// way back.
template <typename VT>
__device__ __forceinline__ void loose_values(const VT* x, int n, float2* out) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int e = threadIdx.x % 32 + j * 32;
    elem(out, j) = e < n ? widen<VT>(x[e]) : 0.f;
  }
}
__device__ __forceinline__ void loose_codes(uint8_t* x, int n, uint2 c) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int e = threadIdx.x % 32 + j * 32;
    if (e < n) x[e] = (uint8_t)((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
  }
}

template <typename VT, int CAP>
__global__ void __launch_bounds__(kThreads, kPackCtas) state8_pack(const __grid_constant__ MomentParamsT<CAP> p) {
  const TileWalk walk = tile_walk(p);
  int t = walk.first;
  if (t >= walk.end) return;
  int hop = 1;
  const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  Place8 cur = place_values(p, t, find_seg(p, t));
  Values8<VT> x;
  if constexpr (kPackAhead<VT>) load_values(p, cur, x);
  for (;;) {
    if constexpr (!kPackAhead<VT>) load_values(p, cur, x);
    t += p.stride;
    const bool more = t < walk.end;
    Place8 next = cur;
    Values8<VT> y;
    if (more) {
      next = place_values(p, t, next_seg(p, cur.si, t, hop));
      if constexpr (kPackAhead<VT>) load_values(p, next, y);
    }
    const MomentSeg& sg = p.seg[cur.si];
    const int n = cur.n - (int)(warp * kMomentBlock);  // of the warp's block
    if (n > 0) {
      const bool whole = whole_block(sg, cur);
      const int64_t block = cur.first + warp * kMomentBlock;
      float2 f[4];
      uint32_t s;
      if (sg.m) {
        if (whole)
          Eight<VT>::widen8(x.m, f);
        else
          loose_values(static_cast<const VT*>(sg.m) + block, n, f);
        const uint2 c = pack_m_values(f, s);
        if (whole)
          __stcs(reinterpret_cast<uint2*>(at_offset(sg.mc + cur.first, threadIdx.x * 8)), c);
        else
          loose_codes(sg.mc + block, n, c);
        if (lane == 0) *at_offset(sg.ms + cur.first / kMomentBlock, warp) = (uint8_t)s;
      }
      if (sg.v) {
        if (whole)
          Eight<VT>::widen8(x.v, f);
        else
          loose_values(static_cast<const VT*>(sg.v) + block, n, f);
        const uint2 c = pack_v_values(f, s);
        if (whole)
          __stcs(reinterpret_cast<uint2*>(at_offset(sg.vc + cur.first, threadIdx.x * 8)), c);
        else
          loose_codes(sg.vc + block, n, c);
        if (lane == 0) *at_offset(sg.vs + cur.first / kMomentBlock, warp) = (uint8_t)s;
      }
    }
    if (!more) break;
    cur = next;
    if constexpr (kPackAhead<VT>) x = y;
  }
}

// Sixteen values (of two words of codes each) to memory.
template <typename VT>
__device__ __forceinline__ void store16(VT* p, const float2* lo, const float2* hi);
template <>
__device__ __forceinline__ void store16<float>(float* p, const float2* lo, const float2* hi) {
  store8(p, lo);
  store8(p + 8, hi);
}
template <>
__device__ __forceinline__ void store16<__nv_bfloat16>(__nv_bfloat16* p, const float2* lo, const float2* hi) {
  float2 w[4];  // pairs of bf16, moved as the bits they are
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    // the values are exact in bf16: their upper halves are the rounding
    const float2* x = k < 2 ? lo + 2 * k : hi + 2 * (k - 2);
    w[k].x = __uint_as_float(__byte_perm(__float_as_uint(x[0].x), __float_as_uint(x[0].y), 0x7632));
    w[k].y = __uint_as_float(__byte_perm(__float_as_uint(x[1].x), __float_as_uint(x[1].y), 0x7632));
  }
  store8(reinterpret_cast<float*>(p), w);
}

__device__ __forceinline__ float widen_m1(uint8_t code, uint32_t s) {
  return __fmul_rn(__half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3))), m_unit(s));
}
__device__ __forceinline__ float widen_v1(uint32_t code, uint32_t s) {
  return __uint_as_float(s == 255u ? 0x7FC00000u : code ? (s << 23) + (code << 20) : 0u);
}

// Sixteen elements per thread, which lie in one block.  A thread loads its
// next tile's codes before it widens and stores this one's.  Bound by memory
// at this mix of one byte read per two or four written: at 1.35e9 elements
// 1160 us to bf16 and 1928 to fp32, 6.96 and 6.98 TB/s, with walks of two
// rounds; 1268 and 2198 without a limit (see launch_walk).  Two to four CTAs
// per SM are alike, six 3 % slower; fp32 stores of 1 KB runs per warp 1 %.
constexpr int kUnpackRounds = 2;
struct Codes16 {
  uint4 m, v;
  uint32_t ms, vs;
};
struct UnpackPlace {
  int si;
  int64_t first;
  int n;
  bool full;  // the thread's elements are in the tensor, on vector boundaries
};
template <typename P>
__device__ __forceinline__ UnpackPlace place_codes(const P& p, int t, int si) {
  const MomentSeg& sg = p.seg[si];
  UnpackPlace a;
  a.si = si;
  a.first = (int64_t)(t - sg.tile0) * kUnpackTile;
  a.n = (int)min((int64_t)kUnpackTile, sg.len - a.first);
  if (!DOPT_TILE_OK(p, kSiteListMoments, a.first, a.n, sg.len)) a.n = 0;
  a.full = sg.vec && (int)(threadIdx.x * 16 + 16) <= a.n;
  return a;
}
template <typename P>
__device__ __forceinline__ void load_codes16(const P& p, const UnpackPlace& a, Codes16& c) {
  if (!a.full) return;
  const MomentSeg& sg = p.seg[a.si];
  const uint32_t e = threadIdx.x * 16;
  if (sg.m) {
    c.m = __ldcs(reinterpret_cast<const uint4*>(at_offset(sg.mc + a.first, e)));
    c.ms = *at_offset(sg.ms + a.first / kMomentBlock, e / kMomentBlock);
  }
  if (sg.v) {
    c.v = __ldcs(reinterpret_cast<const uint4*>(at_offset(sg.vc + a.first, e)));
    c.vs = *at_offset(sg.vs + a.first / kMomentBlock, e / kMomentBlock);
  }
}

template <typename VT, int CAP>
__global__ void __launch_bounds__(kThreads, 4) state8_unpack(const __grid_constant__ MomentParamsT<CAP> p) {
  static_assert(kUnpackTile == kThreads * 16 && kMomentBlock % 16 == 0, "sixteen elements per thread");
  const TileWalk walk = tile_walk(p);
  int t = walk.first;
  if (t >= walk.end) return;
  int hop = 1;
  UnpackPlace cur = place_codes(p, t, find_seg(p, t));
  Codes16 c;
  load_codes16(p, cur, c);
  for (;;) {
    t += p.stride;
    const bool more = t < walk.end;
    UnpackPlace next = cur;
    Codes16 d;
    if (more) {
      next = place_codes(p, t, next_seg(p, cur.si, t, hop));
      load_codes16(p, next, d);
    }
    const MomentSeg& sg = p.seg[cur.si];
    const uint32_t e = threadIdx.x * 16;
    if (cur.full) {
      float2 lo[4], hi[4];
      if (sg.m) {
        const float2 unit = both(m_unit(c.ms));
        widen_m(make_uint2(c.m.x, c.m.y), lo);
        widen_m(make_uint2(c.m.z, c.m.w), hi);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          lo[k] = __fmul2_rn(lo[k], unit);
          hi[k] = __fmul2_rn(hi[k], unit);
        }
        store16<VT>(at_offset(static_cast<VT*>(sg.m) + cur.first, e), lo, hi);
      }
      if (sg.v) {
        widen_v(make_uint2(c.v.x, c.v.y), c.vs, lo);
        widen_v(make_uint2(c.v.z, c.v.w), c.vs, hi);
        store16<VT>(at_offset(static_cast<VT*>(sg.v) + cur.first, e), lo, hi);
      }
    } else if (!sg.vec) {
      // arrays with no common vector boundary: consecutive lanes take
      // consecutive elements, four loads at a time
#pragma unroll 1
      for (uint32_t j0 = 0; j0 < 16; j0 += 4) {
        uint8_t cm[4], cv[4], sm[4], sv[4];
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
          const uint32_t i = threadIdx.x + (j0 + j) * kThreads;
          const bool in = (int)i < cur.n;
          const int64_t at = cur.first + i, block = cur.first / kMomentBlock + i / kMomentBlock;
          cm[j] = in && sg.m ? sg.mc[at] : 0;
          sm[j] = in && sg.m ? sg.ms[block] : 0;
          cv[j] = in && sg.v ? sg.vc[at] : 0;
          sv[j] = in && sg.v ? sg.vs[block] : 0;
        }
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
          const uint32_t i = threadIdx.x + (j0 + j) * kThreads;
          if ((int)i >= cur.n) continue;
          if (sg.m) static_cast<VT*>(sg.m)[cur.first + i] = narrow<VT>(widen_m1(cm[j], sm[j]));
          if (sg.v) static_cast<VT*>(sg.v)[cur.first + i] = narrow<VT>(widen_v1(cv[j], sv[j]));
        }
      }
    }
    // a tensor's ragged end, fewer than sixteen elements: one per thread
    const int tail = (cur.n & ~15) + (int)threadIdx.x;
    if (sg.vec && tail < cur.n) {
      const int64_t at = cur.first + tail;
      if (sg.m) static_cast<VT*>(sg.m)[at] = narrow<VT>(widen_m1(sg.mc[at], sg.ms[at / kMomentBlock]));
      if (sg.v) static_cast<VT*>(sg.v)[at] = narrow<VT>(widen_v1(sg.vc[at], sg.vs[at / kMomentBlock]));
    }
    if (!more) break;
    cur = next;
    c = d;
  }
}

// Launches a pack or unpack kernel's walk, with the compact table where it fits.
template <auto Small, auto Big, int ROUNDS>
int launch_moments(MomentParamsT<kMomentCap>& p, cudaStream_t s, const char* what) {
  if (p.n_seg <= kMomentSmallCap) {
    MomentParamsT<kMomentSmallCap> small = compact_table<MomentParamsT<kMomentSmallCap>, MomentHead>(p);
    return launch_walk<Small, 0, ROUNDS>(small, s, what, false);
  }
  return launch_walk<Big, 0, ROUNDS>(p, s, what, false);
}
template <typename VT>
int launch_pack_t(MomentParamsT<kMomentCap>& p, cudaStream_t s) {
  return launch_moments<state8_pack<VT, kMomentSmallCap>, state8_pack<VT, kMomentCap>, kPackRounds>(p, s, "state8_pack launch");
}
template <typename VT>
int launch_unpack_t(MomentParamsT<kMomentCap>& p, cudaStream_t s) {
  return launch_moments<state8_unpack<VT, kMomentSmallCap>, state8_unpack<VT, kMomentCap>, kUnpackRounds>(
      p, s, "state8_unpack launch");
}

int launch_state8_pack(int32_t values_dtype, MomentParamsT<kMomentCap>& p, cudaStream_t s) {
  return values_dtype == DOPT_F32 ? launch_pack_t<float>(p, s) : launch_pack_t<__nv_bfloat16>(p, s);
}
int launch_state8_unpack(int32_t values_dtype, MomentParamsT<kMomentCap>& p, cudaStream_t s) {
  return values_dtype == DOPT_F32 ? launch_unpack_t<float>(p, s) : launch_unpack_t<__nv_bfloat16>(p, s);
}

}  // namespace dopt
