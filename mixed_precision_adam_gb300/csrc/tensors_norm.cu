// tensors_norm.cu -- the grad norm over a list of tensors: one pass over the
// grads, sum of squares, non-finite flag and zero count per CTA, and the
// finalize (norm, clip coefficient, skip decision) in the last CTA.
//
// Mathematics: sum (g * inv_scale)^2.  A thread adds the squares of 16
// elements in fp32 (a chunk; all terms positive, so at most 16 roundings
// relative to the chunk), chunks by TwoSum into a pair of fp32 words (the
// error-free addition of Ogita, Rump & Oishi, "Accurate sum and dot
// product", SIAM J. Sci. Comput. 2005), threads and CTAs in fp64.  A chunk
// whose sum leaves [2^-90, 2^80] is squared again in fp64, out of line: that
// covers overflow, underflow, infinities and NaN, so the fast path needs
// no test per element.  fp64 per element, or a conversion per chunk, would
// be bound by GB300's fp64 rate.
#include "tensors.cuh"

namespace dopt {

constexpr int kNormVecs = 4;  // 16-byte loads per thread and tile, all in flight together

template <typename GT>
__device__ __forceinline__ void widen_word(uint32_t w, float* x);  // the one or two elements of a 32-bit word
template <>
__device__ __forceinline__ void widen_word<float>(uint32_t w, float* x) { x[0] = __uint_as_float(w); }
template <>
__device__ __forceinline__ void widen_word<__nv_bfloat16>(uint32_t w, float* x) {
  x[0] = __uint_as_float(w << 16);
  x[1] = __uint_as_float(w & 0xFFFF0000u);
}
template <>
__device__ __forceinline__ void widen_word<__half>(uint32_t w, float* x) {
  x[0] = __half2float(__ushort_as_half((unsigned short)(w & 0xFFFFu)));
  x[1] = __half2float(__ushort_as_half((unsigned short)(w >> 16)));
}

// A chunk: 16 elements, in 2 (16-bit) or 4 (fp32) vectors.
template <typename GT>
struct ChunkOf {
  uint4 r[sizeof(GT)];
};

template <typename GT, typename F>
__device__ __forceinline__ void each_of(const ChunkOf<GT>& c, F&& f) {
  constexpr int kPer = 4 / sizeof(GT);
#pragma unroll
  for (int k = 0; k < (int)sizeof(GT); ++k) {
    const uint32_t w[4] = {c.r[k].x, c.r[k].y, c.r[k].z, c.r[k].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x[2];
      widen_word<GT>(w[j], x);
#pragma unroll
      for (int i = 0; i < kPer; ++i) f(x[i]);
    }
  }
}

// Squares of a chunk whose fp32 sum over- or underflowed, in fp64.
template <typename GT>
__device__ __noinline__ double chunk_wide(ChunkOf<GT> c, float inv) {
  double d = 0.0;
  each_of<GT>(c, [&](float x) {
    const double y = __fmul_rn(x, inv);
    d += y * y;
  });
  return d;
}

struct NormSum {
  float s = 0.f, c = 0.f;  // chunks, and the errors of their additions
  double wide = 0.0;       // chunks outside the fast range
  int zeros = 0;
  template <typename GT>
  __device__ __forceinline__ void add(const ChunkOf<GT>& ch, float inv) {
    float q = 0.f;
    int z = 0;
    each_of<GT>(ch, [&](float x) {
      x = __fmul_rn(x, inv);
      z += x == 0.f;
      q = fmaf(x, x, q);
    });
    zeros += z;
    if (!(q <= 0x1p80f) || (q < 0x1p-90f && z < 16)) {
      wide += chunk_wide<GT>(ch, inv);
      q = 0.f;
    }
    const float t = __fadd_rn(s, q), b = __fsub_rn(t, s);  // s stays below 2^80 times a thread's chunks
    c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(q, b)));
    s = t;
  }
};

// One tile: kNormVecs vectors per thread.  Tiles are cut on the 16-byte grid
// of the addresses (sg.shift elements before the tensor's first), so only a
// tensor's first and last vector can be partial, whatever its alignment.
template <typename GT>
__device__ __forceinline__ void norm_tile(const NormSeg& sg, int t, float inv, NormSum& acc) {
  constexpr int kPer = 16 / sizeof(GT), kChunks = kNormVecs / (int)sizeof(GT);
  constexpr int kTile = kNormTileBytes / (int)sizeof(GT);
  static_assert(kNormTileBytes == kThreads * kNormVecs * 16, "a tile is the CTA's vectors");
  const int64_t first = (int64_t)(t - sg.tile0) * kTile - sg.shift;
  const GT* g = static_cast<const GT*>(sg.grad);
  ChunkOf<GT> ch[kChunks];
  uint4* r = &ch[0].r[0];
  if (first >= 0 && first + kTile <= sg.len) {
    const uint4* p = reinterpret_cast<const uint4*>(g + first) + threadIdx.x;
#pragma unroll
    for (int u = 0; u < kNormVecs; ++u) r[u] = __ldcg(p + u * kThreads);
  } else {
#pragma unroll
    for (int u = 0; u < kNormVecs; ++u) {
      const int64_t e = first + (int64_t)(u * kThreads + threadIdx.x) * kPer;
      r[u] = make_uint4(0u, 0u, 0u, 0u);
      if (e >= 0 && e + kPer <= sg.len) {
        r[u] = __ldcg(reinterpret_cast<const uint4*>(g + e));
      } else {
        alignas(16) GT x[kPer];
        *reinterpret_cast<uint4*>(x) = r[u];
        for (int j = 0; j < kPer; ++j) {
          if (e + j >= 0 && e + j < sg.len)
            x[j] = g[e + j];
          else
            --acc.zeros;  // the filling counts as zeros below
        }
        r[u] = *reinterpret_cast<const uint4*>(x);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kChunks; ++k) acc.add<GT>(ch[k], inv);
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) tensors_norm(const __grid_constant__ NormParamsT<CAP> p) {
  NormSum acc;
  int si = 0;
  if ((int)blockIdx.x < p.n_tiles) si = find_seg(p, blockIdx.x);
  for (int t = blockIdx.x; t < p.n_tiles; t += gridDim.x) {
    si = next_seg(p, si, t);
    const NormSeg& sg = p.seg[si];
    if (sg.dtype == DOPT_F32)
      norm_tile<float>(sg, t, p.inv_scale, acc);
    else if (sg.dtype == DOPT_BF16)
      norm_tile<__nv_bfloat16>(sg, t, p.inv_scale, acc);
    else
      norm_tile<__half>(sg, t, p.inv_scale, acc);
  }
  allow_dependent_launch();
  __shared__ double s_sum[kThreads / 32];
  __shared__ int s_zero[kThreads / 32];
  double sum = acc.wide + ((double)acc.s + (double)acc.c);
  int zeros = acc.zeros;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    zeros += __shfl_xor_sync(0xFFFFFFFFu, zeros, o);
  }
  if (threadIdx.x % 32 == 0) {
    s_sum[threadIdx.x / 32] = sum;
    s_zero[threadIdx.x / 32] = zeros;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kThreads / 32; ++i) {
      s_sum[0] += s_sum[i];
      s_zero[0] += s_zero[i];
    }
    p.partials[blockIdx.x] = Partial{s_sum[0], isfinite(s_sum[0]) ? 0 : 1, s_zero[0]};
  }
  if (!p.fin_counter) return;
  __shared__ int s_last;
  if (threadIdx.x == 0) {
    __threadfence();  // this CTA's partial before its ticket
    s_last = atomicAdd(p.fin_counter, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  finalize_call(p.fin);
}

int tensors_norm_grid(int n_seg, int n_tiles, int* grid) {
  return n_seg <= kNormSmallCap ? grid_for(tensors_norm<kNormSmallCap>, n_tiles, grid)
                                : grid_for(tensors_norm<kNormCap>, n_tiles, grid);
}

int launch_tensors_norm(const NormParamsT<kNormCap>& p, cudaStream_t s, int* grid) {
  if (p.n_seg <= kNormSmallCap)
    return launch_table(tensors_norm<kNormSmallCap>, compact_table<NormParamsT<kNormSmallCap>, NormHead>(p), p.n_tiles,
                        s, "tensors_norm launch", grid);
  return launch_table(tensors_norm<kNormCap>, p, p.n_tiles, s, "tensors_norm launch", grid);
}

}  // namespace dopt
