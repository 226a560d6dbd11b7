// tensors_adamw.cu -- AdamW over a list of tensors, moments in fp32.
//
// One pass: reads grad, weight, m and v of every element once, writes
// weight, m, v and the 16-bit param once (28 bytes per element with bf16
// grads and params, 30 with fp32 grads, 28 for fp32 params): bound by
// memory.  A CTA strides over the list's tiles; a thread has four elements
// of a tile, and loads its next tile's before it computes and stores this
// one's, so the memory pipe stays busy under the arithmetic.  Measured on
// 1.35e9 bf16 params with fp32 grads: 5.83 ms, 6.93 TB/s (1.02 of the copy
// bandwidth; 6.09 ms without a limit to a CTA's walk, but 582 us against 590
// on 1.3e8 fp16 ones at odd offsets); fp16 ones with fp16 grads: 5.6 ms, 6.7 TB/s.
// Tensors whose arrays share no vector boundary go by element, with nothing
// loaded ahead of the stores: 1e8 bf16 elements 704 to 724 us against 430.
#include "tensors.cuh"

namespace dopt {

constexpr int kRounds32 = 24;  // of a CTA's walk over the tiles (see launch_walk)

// Four elements of a 16-bit type, as loaded and stored at once.
__device__ __forceinline__ float half_bits(unsigned bits) { return __half2float(__ushort_as_half((unsigned short)bits)); }
__device__ __forceinline__ void widen4(const uint4& r, int dtype, float* x) {
  if (dtype == DOPT_F32) {
    x[0] = __uint_as_float(r.x); x[1] = __uint_as_float(r.y); x[2] = __uint_as_float(r.z); x[3] = __uint_as_float(r.w);
  } else if (dtype == DOPT_BF16) {
    x[0] = __uint_as_float(r.x << 16); x[1] = __uint_as_float(r.x & 0xFFFF0000u);
    x[2] = __uint_as_float(r.y << 16); x[3] = __uint_as_float(r.y & 0xFFFF0000u);
  } else {
    x[0] = half_bits(r.x & 0xFFFFu); x[1] = half_bits(r.x >> 16);
    x[2] = half_bits(r.y & 0xFFFFu); x[3] = half_bits(r.y >> 16);
  }
}
__device__ __forceinline__ uint2 narrow4(int dtype, const float* x) {
  if (dtype == DOPT_BF16) {
    const unsigned a = __bfloat16_as_ushort(__float2bfloat16_rn(x[0])), b = __bfloat16_as_ushort(__float2bfloat16_rn(x[1]));
    const unsigned c = __bfloat16_as_ushort(__float2bfloat16_rn(x[2])), d = __bfloat16_as_ushort(__float2bfloat16_rn(x[3]));
    return make_uint2(a | (b << 16), c | (d << 16));
  }
  const unsigned a = __half_as_ushort(__float2half_rn(x[0])), b = __half_as_ushort(__float2half_rn(x[1]));
  const unsigned c = __half_as_ushort(__float2half_rn(x[2])), d = __half_as_ushort(__float2half_rn(x[3]));
  return make_uint2(a | (b << 16), c | (d << 16));
}

// A thread's part of a tile.  `e` is its first element; `full`: its four
// elements are in the tensor and every array has them on a vector boundary.
struct AdamPart {
  uint4 g;  // as loaded: 16-bit grads take two words
  float4 w, m, v;
  int64_t first;
  int64_t e;
  int si;
  float decay;
  bool full;
};

template <typename P>
__device__ __forceinline__ void place_part(const P& p, int t, int si, AdamPart& a) {
  const AdamSeg& sg = p.seg[si];
  a.si = si;
  // tiles are cut `shift` elements below the first one, where every array
  // that can be read in vectors has a vector boundary
  a.first = (int64_t)(t - sg.tile0) * kAdamTile32 - max(sg.shift, 0);
  a.e = a.first + threadIdx.x * 4;
  a.full = sg.shift >= 0 && a.e >= 0 && a.e + 4 <= sg.len;
  if (!DOPT_TILE_OK(p, kSiteListAdam, a.first + max(sg.shift, 0), 1, sg.len + max(sg.shift, 0))) {
    a.e = a.first = sg.len;  // no elements
    a.full = false;
  }
}
template <typename P>
__device__ __forceinline__ void load_state(const P& p, AdamPart& a) {
  if (!a.full) return;
  const AdamSeg& sg = p.seg[a.si];
  a.w = __ldcs(reinterpret_cast<const float4*>(sg.weight + a.e));
  a.m = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(sg.m) + a.e));
  a.v = __ldcs(reinterpret_cast<const float4*>(static_cast<const float*>(sg.v) + a.e));
}
template <typename P>
__device__ __forceinline__ void load_grad(const P& p, AdamPart& a) {
  if (!a.full) return;
  const AdamSeg& sg = p.seg[a.si];
  if (sg.grad_dtype == DOPT_F32) {
    a.g = __ldcs(reinterpret_cast<const uint4*>(static_cast<const float*>(sg.grad) + a.e));
  } else {
    const uint2 r = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(sg.grad) + a.e));
    a.g.x = r.x;
    a.g.y = r.y;
  }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, 4) tensors_adamw(const __grid_constant__ AdamParamsT<CAP> p) {
  const TileWalk walk = tile_walk(p);
  int t = walk.first;
  const bool work = t < walk.end;
  int hop = 1;
  AdamPart cur;
  if (work) {
    place_part(p, t, find_seg(p, t), cur);
    if (p.early) load_state(p, cur);  // the launch before writes none of it
  }
  wait_for_prior_grids();
  if (!work || (p.found_inf && *p.found_inf)) return;
  AdamScalars s;
  s.c = p.coef ? *p.coef : 1.f;
  s.step_size = p.dev ? p.dev->step_size : p.step_size;
  s.bc2_sqrt = p.dev ? p.dev->bc2_sqrt : p.bc2_sqrt;
  load_grad(p, cur);
  if (!p.early) load_state(p, cur);
  cur.decay = decay_of_seg(p, p.seg[cur.si]);
  for (;;) {
    AdamPart nxt;
    const int tn = t + p.stride;
    const bool more = tn < walk.end;
    if (more) {
      place_part(p, tn, next_seg(p, cur.si, tn, hop), nxt);
      load_grad(p, nxt);
      load_state(p, nxt);
      nxt.decay = nxt.si == cur.si ? cur.decay : decay_of_seg(p, p.seg[nxt.si]);
    }
    const AdamSeg& sg = p.seg[cur.si];
    s.decay = cur.decay;
    float* const wp = sg.weight;
    float* const mp = static_cast<float*>(sg.m);
    float* const vp = static_cast<float*>(sg.v);
    if (cur.full) {
      float g[4];
      widen4(cur.g, sg.grad_dtype, g);
      float w[4] = {cur.w.x, cur.w.y, cur.w.z, cur.w.w};
      float m[4] = {cur.m.x, cur.m.y, cur.m.z, cur.m.w};
      float v[4] = {cur.v.x, cur.v.y, cur.v.z, cur.v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) adamw_element(g[j], p, s, w[j], m[j], v[j]);
      __stcs(reinterpret_cast<float4*>(wp + cur.e), make_float4(w[0], w[1], w[2], w[3]));
      __stcs(reinterpret_cast<float4*>(mp + cur.e), make_float4(m[0], m[1], m[2], m[3]));
      __stcs(reinterpret_cast<float4*>(vp + cur.e), make_float4(v[0], v[1], v[2], v[3]));
      if (sg.param_dtype != DOPT_F32)
        __stcs(reinterpret_cast<uint2*>(static_cast<uint16_t*>(sg.param) + cur.e), narrow4(sg.param_dtype, w));
    } else {
      // a tensor's ragged ends (its own four elements), or a tensor whose
      // arrays have no common vector boundary (consecutive threads take
      // consecutive elements)
      const bool ends = sg.shift >= 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t e = ends ? cur.e + j : cur.first + j * kThreads + threadIdx.x;
        if (e < 0 || e >= sg.len) continue;
        float w = wp[e], m = mp[e], v = vp[e];
        adamw_element(load_element(sg.grad, e, sg.grad_dtype), p, s, w, m, v);
        wp[e] = w;
        mp[e] = m;
        vp[e] = v;
        store_param(sg.param, e, sg.param_dtype, w);
      }
    }
    if (!more) break;
    cur = nxt;
    t = tn;
  }
}

int launch_tensors_adamw(AdamParamsT<kAdamCap>& p, cudaStream_t s) {
  const char* what = "tensors_adamw launch";
  if (p.n_seg <= kAdamSmallCap) {
    AdamParamsT<kAdamSmallCap> small = compact_table<AdamParamsT<kAdamSmallCap>, AdamHead>(p);
    return launch_walk<tensors_adamw<kAdamSmallCap>, 0, kRounds32>(small, s, what, true);
  }
  return launch_walk<tensors_adamw<kAdamCap>, 0, kRounds32>(p, s, what, true);
}

}  // namespace dopt
