// tensors_adamw8.cu -- AdamW over a list of tensors with the moments in 8
// bits, and the moments' conversion between values and 8-bit codes.
#include <cuda_fp8.h>

#include "tensors.cuh"

namespace dopt {

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
// Eight consecutive elements of a type, as loaded and stored at once.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  struct Raw {
    float4 a, b;
  };
  static __device__ __forceinline__ Raw load(const float* p) {
    return Raw{__ldcs(reinterpret_cast<const float4*>(p)), __ldcs(reinterpret_cast<const float4*>(p) + 1)};
  }
  static __device__ __forceinline__ void widen8(const Raw& r, float* x) {
    x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w;
    x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float* x) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(x[0], x[1], x[2], x[3]));
    __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(x[4], x[5], x[6], x[7]));
  }
};
template <>
struct Eight<__nv_bfloat16> {
  using Raw = uint4;
  static __device__ __forceinline__ Raw load(const __nv_bfloat16* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }
  static __device__ __forceinline__ void widen8(const Raw& r, float* x) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = __uint_as_float(w[k] << 16);
      x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  }
};
template <>
struct Eight<__half> {
  using Raw = uint4;
  static __device__ __forceinline__ Raw load(const __half* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }
  static __device__ __forceinline__ void widen8(const Raw& r, float* x) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
      x[2 * k] = f.x;
      x[2 * k + 1] = f.y;
    }
  }
  static __device__ __forceinline__ void store(__half* p, const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __half2 h = __floats2half2_rn(x[2 * k], x[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
  }
};

// Two e4m3 codes as floats, and back.
__device__ __forceinline__ float2 widen_e4m3x2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
  return __half22float2(__half2(h));
}
__device__ __forceinline__ uint32_t narrow_e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// A warp's block of moments: eight codes per lane in two words each.
__device__ __forceinline__ void unpack_block(uint2 mc, uint2 vc, uint32_t ms, uint32_t vs, float* m, float* v) {
  const float unit = m_unit(ms);
  const uint32_t base = vs << 23;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t mw = k < 2 ? mc.x : mc.y;
    const float2 f = widen_e4m3x2((k & 1) ? mw >> 16 : mw & 0xFFFFu);
    m[2 * k] = __fmul_rn(f.x, unit);
    m[2 * k + 1] = __fmul_rn(f.y, unit);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t w = j < 4 ? vc.x : vc.y;
    const int at = 8 * (j & 3);  // the code's bits, moved to 20..27
    const uint32_t c = (at <= 20 ? w << (20 - at) : w >> (at - 20)) & 0x0FF00000u;
    v[j] = __uint_as_float(min(c, 1u) * base + c);  // code 0 is zero
  }
  if (vs == 255u) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(0x7FC00000u);
  }
}

// The largest of a lane's eight |m| or v over the warp, as fp32 bits (the
// order of non-negative floats, NaN above all).
__device__ __forceinline__ uint32_t block_top(const float* x) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
  return __reduce_max_sync(0xFFFFFFFFu, top);
}

__device__ __forceinline__ uint2 pack_m_block(const float* m, uint32_t s) {
  const float up = __uint_as_float((254u - s) << 23);
  uint32_t h[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) h[k] = narrow_e4m3x2(__fmul_rn(m[2 * k], up), __fmul_rn(m[2 * k + 1], up));
  return s == 255u ? make_uint2(0u, 0u) : make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}
// r20: the elements' rounding addends.  The scale keeps codes at most 255.
__device__ __forceinline__ uint2 pack_v_block(const float* v, uint32_t s, const uint32_t* r20) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t b = __float_as_uint(v[j]);
    const int c = max((int)(b + r20[j] - (s << 23)) >> 20, (int)min(b, 1u));  // at least 1 but for zero
    w[j / 4] |= (uint32_t)c << (8 * (j & 3));
  }
  return s == 255u ? make_uint2(0u, 0u) : make_uint2(w[0], w[1]);
}

// A lane's part of a block.  `full`: its eight elements are consecutive, in
// the tensor, and every array has them on a vector boundary.
template <typename GT>
struct Part8 {
  typename Eight<GT>::Raw g;
  typename Eight<float>::Raw w;
  uint2 m, v;
  uint32_t ms, vs;
  int64_t block;  // the block's first element; < 0: none (past the tensor's end)
  int si;
  float decay;
  bool full;
};

template <typename GT, typename P>
__device__ __forceinline__ void place_part(const P& p, int t, int si, Part8<GT>& a) {
  const AdamSeg& sg = p.seg[si];
  a.si = si;
  a.block = (int64_t)(t - sg.tile0) * kAdamTile + (threadIdx.x / 32) * kMomentBlock;
  if (a.block >= sg.len) a.block = -1;
  a.full = sg.shift == 0 && a.block >= 0 && a.block + (threadIdx.x % 32) * 8 + 8 <= sg.len;
}
template <typename GT, typename P>
__device__ __forceinline__ void load_state(const P& p, Part8<GT>& a) {
  const AdamSeg& sg = p.seg[a.si];
  if (a.block >= 0) {
    a.ms = sg.m_scale[a.block / kMomentBlock];
    a.vs = sg.v_scale[a.block / kMomentBlock];
  }
  if (a.full) {
    const int64_t e = a.block + (threadIdx.x % 32) * 8;
    a.w = Eight<float>::load(sg.weight + e);
    a.m = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(sg.m) + e));
    a.v = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(sg.v) + e));
  }
}
template <typename GT, typename P>
__device__ __forceinline__ void load_grad(const P& p, Part8<GT>& a) {
  if (a.full)
    a.g = Eight<GT>::load(static_cast<const GT*>(p.seg[a.si].grad) + a.block + (threadIdx.x % 32) * 8);
}

// Updates a lane's part (whole warps: the block's scales are reduced over it).
template <typename PT, typename GT>
__device__ __forceinline__ void step_part(const AdamHead& p, const AdamSeg& sg, const Part8<GT>& a,
                                          const AdamScalars& s, uint32_t key) {
  const int lane = threadIdx.x % 32;
  float* const wp = sg.weight + a.block;
  uint8_t* const mp = static_cast<uint8_t*>(sg.m) + a.block;
  uint8_t* const vp = static_cast<uint8_t*>(sg.v) + a.block;
  const GT* const gp = static_cast<const GT*>(sg.grad) + a.block;
  PT* const pp = static_cast<PT*>(sg.param) + a.block;
  // element j of the lane: consecutive where the tensor is read in vectors,
  // 32 apart (consecutive lanes, consecutive elements) where it is not
  const bool vec = sg.shift == 0;
  const int n = (int)min((int64_t)kMomentBlock, sg.len - a.block);
  const int first = vec ? lane * 8 : lane, stride = vec ? 1 : 32;
  float g[8], w[8], m[8], v[8];
  uint2 mc, vc;
  if (a.full) {
    Eight<GT>::widen8(a.g, g);
    Eight<float>::widen8(a.w, w);
    mc = a.m;
    vc = a.v;
  } else {
    uint32_t mw[2] = {0u, 0u}, vw[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = first + j * stride;
      const bool in = e < n;
      g[j] = in ? widen<GT>(gp[e]) : 0.f;
      w[j] = in ? wp[e] : 0.f;
      mw[j / 4] |= (in ? (uint32_t)mp[e] : 0u) << (8 * (j & 3));
      vw[j / 4] |= (in ? (uint32_t)vp[e] : 0u) << (8 * (j & 3));
    }
    mc = make_uint2(mw[0], mw[1]);
    vc = make_uint2(vw[0], vw[1]);
  }
  unpack_block(mc, vc, a.ms, a.vs, m, v);
#pragma unroll
  for (int j = 0; j < 8; ++j) adamw_element(g[j], p, s, w[j], m[j], v[j]);
  if (a.full) {
    Eight<float>::store(wp + first, w);
    if constexpr (sizeof(PT) == 2) Eight<PT>::store(pp + first, w);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = first + j * stride;
      if (e < n) {
        wp[e] = w[j];
        if constexpr (sizeof(PT) == 2) pp[e] = narrow<PT>(w[j]);
      } else {
        m[j] = v[j] = 0.f;  // past the end: no part in the scales (NaN blocks)
      }
    }
  }
  const uint32_t ms = m_scale_of(block_top(m)), vs = v_scale_of(block_top(v));
  uint32_t r20[8];
  const uint32_t at = (uint32_t)((uint64_t)a.block >> 1);
  if (vec) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t h = hash_pair((at + lane * 4 + k) * kHashPair + key);
      r20[2 * k] = (h << 4) & 0xFFFF0u;
      r20[2 * k + 1] = (h >> 12) & 0xFFFF0u;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t h = hash_pair((at + (lane >> 1) + j * 16) * kHashPair + key);
      r20[j] = ((lane & 1) ? h >> 12 : h << 4) & 0xFFFF0u;
    }
  }
  mc = pack_m_block(m, ms);
  vc = pack_v_block(v, vs, r20);
  if (lane == 0) {
    sg.m_scale[a.block / kMomentBlock] = (uint8_t)ms;
    sg.v_scale[a.block / kMomentBlock] = (uint8_t)vs;
  }
  if (a.full) {
    __stcs(reinterpret_cast<uint2*>(mp + first), mc);
    __stcs(reinterpret_cast<uint2*>(vp + first), vc);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = first + j * stride;
      if (e < n) {
        mp[e] = (uint8_t)((j < 4 ? mc.x : mc.y) >> (8 * (j & 3)));
        vp[e] = (uint8_t)((j < 4 ? vc.x : vc.y) >> (8 * (j & 3)));
      }
    }
  }
}

template <typename PT, typename GT, int CAP>
__global__ void __launch_bounds__(kThreads, 3) tensors_adamw8(const __grid_constant__ AdamParamsT<CAP> p) {
  int t = blockIdx.x;
  const bool work = t < p.n_tiles;
  Part8<GT> cur;
  if (work) {
    place_part<GT>(p, t, find_seg(p, t), cur);
    if (p.early) load_state<GT>(p, cur);  // the launch before writes none of it
  }
  wait_for_prior_grids();
  if (!work || (p.found_inf && *p.found_inf)) return;
  AdamScalars s;
  s.c = p.coef ? *p.coef : 1.f;
  s.step_size = p.dev ? p.dev->step_size : p.step_size;
  s.bc2_sqrt = p.dev ? p.dev->bc2_sqrt : p.bc2_sqrt;
  const uint32_t key = p.key + (p.d_step ? (uint32_t)*p.d_step * kHashStep : 0u);
  load_grad<GT>(p, cur);
  if (!p.early) load_state<GT>(p, cur);
  cur.decay = decay_of_seg(p, p.seg[cur.si]);
  for (;;) {
    Part8<GT> nxt;
    const int tn = t + (int)gridDim.x;
    const bool more = tn < p.n_tiles;
    if (more) {
      place_part<GT>(p, tn, next_seg(p, cur.si, tn), nxt);
      load_grad<GT>(p, nxt);
      load_state<GT>(p, nxt);
      nxt.decay = nxt.si == cur.si ? cur.decay : decay_of_seg(p, p.seg[nxt.si]);
    }
    s.decay = cur.decay;
    if (cur.block >= 0) step_part<PT, GT>(p, p.seg[cur.si], cur, s, key + p.seg[cur.si].key);
    if (!more) break;
    cur = nxt;
    t = tn;
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

// One warp per block, eight elements per lane: consecutive ones in vectors
// where every array has its first element on a vector boundary, else 32
// apart.  A lane's part of a moment's values and codes:
template <typename VT>
__device__ __forceinline__ void load_values(const VT* x, bool vec, int lane, int n, float* out) {
  if (vec && lane * 8 + 8 <= n) {
    Eight<VT>::widen8(Eight<VT>::load(x + lane * 8), out);
    return;
  }
  const int first = vec ? lane * 8 : lane, stride = vec ? 1 : 32;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int e = first + j * stride;
    out[j] = e < n ? widen<VT>(x[e]) : 0.f;
  }
}
template <typename VT>
__device__ __forceinline__ void store_values(VT* x, bool vec, int lane, int n, const float* in) {
  if (vec && lane * 8 + 8 <= n) {
    Eight<VT>::store(x + lane * 8, in);
    return;
  }
  const int first = vec ? lane * 8 : lane, stride = vec ? 1 : 32;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int e = first + j * stride;
    if (e < n) x[e] = narrow<VT>(in[j]);
  }
}
__device__ __forceinline__ uint2 load_codes(const uint8_t* x, bool vec, int lane, int n) {
  if (vec && lane * 8 + 8 <= n) return __ldcs(reinterpret_cast<const uint2*>(x + lane * 8));
  const int first = vec ? lane * 8 : lane, stride = vec ? 1 : 32;
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int e = first + j * stride;
    if (e < n) w[j / 4] |= (uint32_t)x[e] << (8 * (j & 3));
  }
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes(uint8_t* x, bool vec, int lane, int n, uint2 c) {
  if (vec && lane * 8 + 8 <= n) {
    __stcs(reinterpret_cast<uint2*>(x + lane * 8), c);
    return;
  }
  const int first = vec ? lane * 8 : lane, stride = vec ? 1 : 32;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int e = first + j * stride;
    if (e < n) x[e] = (uint8_t)((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
  }
}

// The blocks of a table's tiles, one per warp: f(tensor, first element,
// elements of the block, the tensor's vector flag).
template <int CAP, typename F>
__device__ __forceinline__ void each_block(const MomentParamsT<CAP>& p, F&& f) {
  int si = -1;
  for (int t = blockIdx.x; t < p.n_tiles; t += gridDim.x) {
    si = si < 0 ? find_seg(p, t) : next_seg(p, si, t);
    const MomentSeg& sg = p.seg[si];
    const int64_t off = (int64_t)(t - sg.tile0) * kAdamTile + (threadIdx.x / 32) * kMomentBlock;
    if (off < sg.len) f(sg, off, (int)min((int64_t)kMomentBlock, sg.len - off), sg.vec != 0);
  }
}

template <typename VT, int CAP>
__global__ void __launch_bounds__(kThreads) state8_pack(const __grid_constant__ MomentParamsT<CAP> p) {
  const int lane = threadIdx.x % 32;
  each_block(p, [&](const MomentSeg& sg, int64_t off, int n, bool vec) {
    float m[8], v[8];
    if (sg.m) load_values(static_cast<const VT*>(sg.m) + off, vec, lane, n, m);
    if (sg.v) load_values(static_cast<const VT*>(sg.v) + off, vec, lane, n, v);
    if (sg.m) {
      const uint32_t s = m_scale_of(block_top(m));
      if (lane == 0) sg.ms[off / kMomentBlock] = (uint8_t)s;
      store_codes(sg.mc + off, vec, lane, n, pack_m_block(m, s));
    }
    if (sg.v) {
      uint32_t nearest[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // -0 is 0; what is below 0 is not a second moment: NaN
        v[j] = v[j] < 0.f ? __uint_as_float(0x7FC00000u) : __fadd_rn(v[j], 0.f);
        nearest[j] = 0x80000u;
      }
      const uint32_t s = v_scale_of(block_top(v));
      if (lane == 0) sg.vs[off / kMomentBlock] = (uint8_t)s;
      store_codes(sg.vc + off, vec, lane, n, pack_v_block(v, s, nearest));
    }
  });
}

template <typename VT, int CAP>
__global__ void __launch_bounds__(kThreads) state8_unpack(const __grid_constant__ MomentParamsT<CAP> p) {
  const int lane = threadIdx.x % 32;
  each_block(p, [&](const MomentSeg& sg, int64_t off, int n, bool vec) {
    uint2 mc = make_uint2(0u, 0u), vc = mc;
    uint32_t ms = 0u, vs = 0u;
    if (sg.m) {
      mc = load_codes(sg.mc + off, vec, lane, n);
      ms = sg.ms[off / kMomentBlock];
    }
    if (sg.v) {
      vc = load_codes(sg.vc + off, vec, lane, n);
      vs = sg.vs[off / kMomentBlock];
    }
    float m[8], v[8];
    unpack_block(mc, vc, ms, vs, m, v);
    if (sg.m) store_values(static_cast<VT*>(sg.m) + off, vec, lane, n, m);
    if (sg.v) store_values(static_cast<VT*>(sg.v) + off, vec, lane, n, v);
  });
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
