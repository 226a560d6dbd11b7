// tensors_adamw8.cu -- AdamW over a list of tensors with the moments in 8
// bits, and the moments' conversion between values and 8-bit codes.
#include <cuda_fp8.h>

#include "tensors.cuh"

namespace dopt {

static_assert(kMomentBlock == 256 && kAdamTile % kMomentBlock == 0, "one warp per block, 8 elements per lane");

__device__ __forceinline__ uint32_t exponent_of(uint32_t bits, uint32_t up) { return (bits + up) >> 23; }

__device__ __forceinline__ float unpack_m(uint8_t code, float unit) {
  return __fmul_rn(__half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3))), unit);
}
__device__ __forceinline__ float m_unit(uint32_t s) {
  return s == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(s << 23);
}
__device__ __forceinline__ float unpack_v(uint32_t code, uint32_t s) {
  const uint32_t zero = s == 255u ? 0x7FC00000u : 0u;
  return __uint_as_float(code ? (s << 23) + (code << 20) : zero);
}

__device__ __forceinline__ uint32_t hash_pair(uint32_t x) {
  uint64_t q = (uint64_t)x * kHashMul1;
  x = (uint32_t)q ^ (uint32_t)(q >> 32);
  q = (uint64_t)x * kHashMul2;
  return (uint32_t)q ^ (uint32_t)(q >> 32);
}

// A block's exp_avg scale from the bits of its largest magnitude; the
// multiplier that brings the block to e4m3's range (0 for a block that is
// not finite).
__device__ __forceinline__ uint32_t m_scale_of(uint32_t top) {
  const uint32_t e = exponent_of(top, 0x1FFFFFu);
  return e >= 255u ? 255u : max((int)e - 8, 8);
}
__device__ __forceinline__ uint32_t v_scale_of(uint32_t top) {
  const uint32_t e = exponent_of(top, 0x0FFFFFu);
  return e >= 255u ? 255u : (uint32_t)max((int)e - 31, 0);
}
__device__ __forceinline__ uint8_t pack_m(float m, uint32_t s) {
  return s == 255u ? 0 : __nv_cvt_float_to_fp8(__fmul_rn(m, __uint_as_float((254u - s) << 23)), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint8_t pack_v(float v, uint32_t s, uint32_t r20) {
  if (s == 255u || v == 0.f) return 0;
  const int c = (int)(__float_as_uint(v) + r20 - (s << 23)) >> 20;
  return (uint8_t)min(max(c, 1), 255);
}

template <typename PT, typename GT, int CAP>
__global__ void __launch_bounds__(kThreads) tensors_adamw8(const __grid_constant__ AdamParamsT<CAP> p) {
  wait_for_prior_grids();
  if (p.found_inf && *p.found_inf) return;
  AdamScalars s;
  s.c = p.coef ? *p.coef : 1.f;
  s.step_size = p.dev ? p.dev->step_size : p.step_size;
  s.bc2_sqrt = p.dev ? p.dev->bc2_sqrt : p.bc2_sqrt;
  const uint32_t step_key = p.key + (p.d_step ? (uint32_t)*p.d_step * kHashStep : 0u);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int si = -1;
  for (int t = blockIdx.x; t < p.n_tiles; t += gridDim.x) {
    const int k = si < 0 ? find_seg(p, t) : next_seg(p, si, t);
    const AdamSeg& sg = p.seg[k];
    if (k != si) s.decay = decay_of_seg(p, sg);
    si = k;
    const int64_t off = (int64_t)(t - sg.tile0) * kAdamTile + warp * kMomentBlock;
    if (off >= sg.len) continue;  // whole warps
    const int n = (int)min((int64_t)kMomentBlock, sg.len - off);
    const int64_t block = off / kMomentBlock;
    const GT* g = static_cast<const GT*>(sg.grad) + off;
    float* w = sg.weight + off;
    uint8_t* mc = static_cast<uint8_t*>(sg.m) + off;
    uint8_t* vc = static_cast<uint8_t*>(sg.v) + off;
    const float mu = m_unit(sg.m_scale[block]);
    const uint32_t vs = sg.v_scale[block];
    float m[8], v[8];
    uint32_t mtop = 0, vtop = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = lane + 32 * j;
      m[j] = v[j] = 0.f;
      if (e < n) {
        float ww = w[e];
        m[j] = unpack_m(mc[e], mu);
        v[j] = unpack_v(vc[e], vs);
        adamw_element(widen<GT>(g[e]), p, s, ww, m[j], v[j]);
        w[e] = ww;
        if constexpr (sizeof(PT) == 2) static_cast<PT*>(sg.param)[off + e] = narrow<PT>(ww);
        mtop = max(mtop, __float_as_uint(m[j]) & 0x7FFFFFFFu);
        vtop = max(vtop, __float_as_uint(v[j]));
      }
    }
    mtop = __reduce_max_sync(0xFFFFFFFFu, mtop);
    vtop = __reduce_max_sync(0xFFFFFFFFu, vtop);
    const uint32_t ms1 = m_scale_of(mtop), vs1 = v_scale_of(vtop);
    if (lane == 0) {
      sg.m_scale[block] = (uint8_t)ms1;
      sg.v_scale[block] = (uint8_t)vs1;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = lane + 32 * j;
      if (e < n) {
        const uint64_t i = (uint64_t)off + e;
        const uint32_t h = hash_pair((uint32_t)(i >> 1) * kHashPair + step_key + sg.key);
        mc[e] = pack_m(m[j], ms1);
        vc[e] = pack_v(v[j], vs1, ((i & 1) ? h >> 16 : h & 0xFFFFu) << 4);
      }
    }
  }
}

template <typename PT, typename GT>
int launch_adamw8_t(const AdamParamsT<kAdamCap>& p, cudaStream_t s) {
  if (p.n_seg <= kAdamSmallCap)
    return launch_table(tensors_adamw8<PT, GT, kAdamSmallCap>, compact_table<AdamParamsT<kAdamSmallCap>, AdamHead>(p),
                        p.n_tiles, s, "tensors_adamw8 launch", nullptr, true);
  return launch_table(tensors_adamw8<PT, GT, kAdamCap>, p, p.n_tiles, s, "tensors_adamw8 launch", nullptr, true);
}

int launch_tensors_adamw8(int32_t param_dtype, int32_t grad_dtype, const AdamParamsT<kAdamCap>& p, cudaStream_t s) {
  const bool f32 = grad_dtype == DOPT_F32;
  switch (param_dtype) {
    case DOPT_BF16: return f32 ? launch_adamw8_t<__nv_bfloat16, float>(p, s) : launch_adamw8_t<__nv_bfloat16, __nv_bfloat16>(p, s);
    case DOPT_F16: return f32 ? launch_adamw8_t<__half, float>(p, s) : launch_adamw8_t<__half, __half>(p, s);
    default: return launch_adamw8_t<float, float>(p, s);
  }
}

// ------------------------------------------------------- pack and unpack --

template <typename VT, int CAP>
__global__ void __launch_bounds__(kThreads) state8_pack(const __grid_constant__ MomentParamsT<CAP> p) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int si = -1;
  for (int t = blockIdx.x; t < p.n_tiles; t += gridDim.x) {
    si = si < 0 ? find_seg(p, t) : next_seg(p, si, t);
    const MomentSeg& sg = p.seg[si];
    const int64_t off = (int64_t)(t - sg.tile0) * kAdamTile + warp * kMomentBlock;
    if (off >= sg.len) continue;
    const int n = (int)min((int64_t)kMomentBlock, sg.len - off);
    const int64_t block = off / kMomentBlock;
    if (sg.m) {
      float x[8];
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = lane + 32 * j;
        x[j] = e < n ? widen<VT>(static_cast<const VT*>(sg.m)[off + e]) : 0.f;
        top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
      }
      const uint32_t s = m_scale_of(__reduce_max_sync(0xFFFFFFFFu, top));
      if (lane == 0) sg.ms[block] = (uint8_t)s;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (lane + 32 * j < n) sg.mc[off + lane + 32 * j] = pack_m(x[j], s);
    }
    if (sg.v) {
      float x[8];
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = lane + 32 * j;
        x[j] = e < n ? __fadd_rn(widen<VT>(static_cast<const VT*>(sg.v)[off + e]), 0.f) : 0.f;  // -0 is 0
        top = max(top, __float_as_uint(x[j]));
      }
      const uint32_t s = v_scale_of(__reduce_max_sync(0xFFFFFFFFu, top));
      if (lane == 0) sg.vs[block] = (uint8_t)s;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (lane + 32 * j < n) sg.vc[off + lane + 32 * j] = pack_v(x[j], s, 0x80000u);
    }
  }
}

template <typename VT, int CAP>
__global__ void __launch_bounds__(kThreads) state8_unpack(const __grid_constant__ MomentParamsT<CAP> p) {
  int si = -1;
  for (int t = blockIdx.x; t < p.n_tiles; t += gridDim.x) {
    si = si < 0 ? find_seg(p, t) : next_seg(p, si, t);
    const MomentSeg& sg = p.seg[si];
    const int64_t off = (int64_t)(t - sg.tile0) * kAdamTile;
    const int n = (int)min((int64_t)kAdamTile, sg.len - off);
    for (int e = threadIdx.x; e < n; e += kThreads) {
      const int64_t i = off + e, block = i / kMomentBlock;
      if (sg.m) static_cast<VT*>(sg.m)[i] = narrow<VT>(unpack_m(sg.mc[i], m_unit(sg.ms[block])));
      if (sg.v) static_cast<VT*>(sg.v)[i] = narrow<VT>(unpack_v(sg.vc[i], sg.vs[block]));
    }
  }
}

template <typename KSmall, typename KBig>
int launch_moments(KSmall small, KBig big, const MomentParamsT<kMomentCap>& p, cudaStream_t s, const char* what) {
  if (p.n_seg <= kMomentSmallCap) {
    MomentParamsT<kMomentSmallCap> q{};
    q.n_seg = p.n_seg;
    q.n_tiles = p.n_tiles;
    for (int i = 0; i < p.n_seg; ++i) q.seg[i] = p.seg[i];
    return launch_table(small, q, p.n_tiles, s, what);
  }
  return launch_table(big, p, p.n_tiles, s, what);
}

int launch_state8_pack(int32_t values_dtype, const MomentParamsT<kMomentCap>& p, cudaStream_t s) {
  if (values_dtype == DOPT_F32)
    return launch_moments(state8_pack<float, kMomentSmallCap>, state8_pack<float, kMomentCap>, p, s, "state8_pack launch");
  return launch_moments(state8_pack<__nv_bfloat16, kMomentSmallCap>, state8_pack<__nv_bfloat16, kMomentCap>, p, s,
                        "state8_pack launch");
}

int launch_state8_unpack(int32_t values_dtype, const MomentParamsT<kMomentCap>& p, cudaStream_t s) {
  if (values_dtype == DOPT_F32)
    return launch_moments(state8_unpack<float, kMomentSmallCap>, state8_unpack<float, kMomentCap>, p, s,
                          "state8_unpack launch");
  return launch_moments(state8_unpack<__nv_bfloat16, kMomentSmallCap>, state8_unpack<__nv_bfloat16, kMomentCap>, p, s,
                        "state8_unpack launch");
}

}  // namespace dopt
