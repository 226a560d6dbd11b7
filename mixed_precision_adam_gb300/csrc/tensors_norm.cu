// tensors_norm.cu -- the grad norm over a list of tensors: one pass over the
// grads, sum of squares, non-finite flag and zero count per CTA, and the
// finalize (norm, clip coefficient, skip decision) in a launch of one CTA
// that starts under it.  (A ticket counter and the finalize in the last CTA,
// as the sharded step has it, needs its counter cleared before every call
// and two fences after: 12.3 us for a 413,856-element list, against 6.5.)
//
// Mathematics: sum (g * inv_scale)^2.  A thread adds the squares of 16
// elements in fp32 (a chunk; all terms positive, so at most 16 roundings
// relative to the chunk), chunks by TwoSum into a pair of fp32 words (the
// error-free addition of Ogita, Rump & Oishi, "Accurate sum and dot
// product", SIAM J. Sci. Comput. 2005), threads and CTAs in fp64.  A chunk
// whose sum leaves [2^-90, 2^80] is squared again in fp64, out of line: that
// covers overflow, underflow, infinities and NaN, so the fast path needs
// no test per element.  fp64 per element, or a conversion per chunk, would
// be bound by GB300's fp64 rate; with packed fp32 pairs and zeros found by a
// running minimum an element takes about 3 issue slots of the 11 that its 2
// bytes allow, and the pass is bound by memory: 1.35e9 bf16 grads in 368 us,
// 7.3 TB/s (1.08 of the copy bandwidth), finalize included.
#include "tensors.cuh"

namespace dopt {

// 32-byte loads per thread and tile, all in flight together, and CTAs per SM:
// four of each keep 128 KB per SM in flight.  Two loads: 5 % slower; more CTAs
// with two loads, 25 % and more (registers); a ring of asynchronous copies in
// shared memory, 43 % (its instructions per 16 bytes bound it).
constexpr int kNormVecs = 4, kNormCtas = 4;
constexpr int kNormTileBytes = kThreads * kNormVecs * 32;

// A chunk: 16 elements, in one (16-bit) or two (fp32) 32-byte vectors.
template <typename GT>
struct ChunkOf {
  uint32_t r[4 * sizeof(GT)];
};
template <typename GT>
constexpr int kChunkVecs = (int)sizeof(GT) / 2;

// Element pair i of a chunk.
template <typename GT>
__device__ __forceinline__ float2 pair_of(const ChunkOf<GT>& c, int i);
template <>
__device__ __forceinline__ float2 pair_of<float>(const ChunkOf<float>& c, int i) {
  return make_float2(__uint_as_float(c.r[2 * i]), __uint_as_float(c.r[2 * i + 1]));
}
template <>
__device__ __forceinline__ float2 pair_of<__nv_bfloat16>(const ChunkOf<__nv_bfloat16>& c, int i) {
  return make_float2(__uint_as_float(c.r[i] << 16), __uint_as_float(c.r[i] & 0xFFFF0000u));
}
template <>
__device__ __forceinline__ float2 pair_of<__half>(const ChunkOf<__half>& c, int i) {
  return __half22float2(*reinterpret_cast<const __half2*>(&c.r[i]));
}

__device__ __forceinline__ float min3_abs(float a, float b, float c) {
  float d;
  asm("min.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Squares of a chunk whose fp32 sum over- or underflowed, in fp64.
template <typename GT>
__device__ __noinline__ double chunk_wide(ChunkOf<GT> c, float inv) {
  double d = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 x = pair_of<GT>(c, i);
    const double a = __fmul_rn(x.x, inv), b = __fmul_rn(x.y, inv);
    d += a * a + b * b;
  }
  return d;
}
// The zeros of a chunk that has one.
template <typename GT>
__device__ __forceinline__ int chunk_zeros(const ChunkOf<GT>& c, float inv) {
  int z = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 x = pair_of<GT>(c, i);
    z += (__fmul_rn(x.x, inv) == 0.f) + (__fmul_rn(x.y, inv) == 0.f);
  }
  return z;
}

struct NormSum {
  float s = 0.f, c = 0.f;  // chunks, and the errors of their additions
  double wide = 0.0;       // chunks outside the fast range
  int zeros = 0;
  template <typename GT>
  __device__ __forceinline__ void add(const ChunkOf<GT>& ch, float2 inv) {
    float2 q2 = make_float2(0.f, 0.f);
    float least = __int_as_float(0x7F800000);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = __fmul2_rn(pair_of<GT>(ch, i), inv);
      least = min3_abs(x.x, x.y, least);
      q2 = __ffma2_rn(x, x, q2);
    }
    float q = __fadd_rn(q2.x, q2.y);
    int z = 0;
    if (least == 0.f) zeros += z = chunk_zeros<GT>(ch, inv.x);
    if (!(q <= 0x1p80f) || (q < 0x1p-90f && z < 16)) {
      wide += chunk_wide<GT>(ch, inv.x);
      q = 0.f;
    }
    const float t = __fadd_rn(s, q), b = __fsub_rn(t, s);  // s stays below 2^80 times a thread's chunks
    c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(q, b)));
    s = t;
  }
};

__device__ __forceinline__ void load32(const void* p, uint32_t* r) {
  asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "l"(p));
}

// One tile: kNormVecs vectors per thread.  Tiles are cut on the 32-byte grid
// of the addresses (sg.shift elements before the tensor's first), so only a
// tensor's first and last vector can be partial, whatever its alignment.
template <typename GT>
__device__ __forceinline__ void norm_tile(const NormSeg& sg, int t, float2 inv, NormSum& acc) {
  constexpr int kPer = 32 / sizeof(GT);  // elements per vector
  constexpr int kTile = kNormTileBytes / (int)sizeof(GT);
  constexpr int kChunks = kNormVecs / kChunkVecs<GT>;
  static_assert(kNormVecs % 2 == 0, "whole fp32 chunks");
  const int64_t first = (int64_t)(t - sg.tile0) * kTile - sg.shift;
  const GT* g = static_cast<const GT*>(sg.grad);
  ChunkOf<GT> ch[kChunks];
  uint32_t* r = &ch[0].r[0];
  if (first >= 0 && first + kTile <= sg.len) {
    const char* p = reinterpret_cast<const char*>(g + first) + threadIdx.x * 32;
#pragma unroll
    for (int u = 0; u < kNormVecs; ++u) load32(p + u * kThreads * 32, r + 8 * u);
  } else {
#pragma unroll
    for (int u = 0; u < kNormVecs; ++u) {
      const int64_t e = first + (int64_t)(u * kThreads + threadIdx.x) * kPer;
      if (e >= 0 && e + kPer <= sg.len) {
        load32(g + e, r + 8 * u);
      } else if (e >= sg.len) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r[8 * u + j] = 0u;
        acc.zeros -= kPer;
      } else {
        alignas(16) GT x[kPer];
        uint32_t* w = reinterpret_cast<uint32_t*>(x);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 0u;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          if (e + j >= 0 && e + j < sg.len)
            x[j] = g[e + j];
          else
            --acc.zeros;  // the filling counts as zeros below
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) r[8 * u + j] = w[j];
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kChunks; ++k) acc.add<GT>(ch[k], inv);
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, kNormCtas) tensors_norm(const __grid_constant__ NormParamsT<CAP> p) {
  NormSum acc;
  const float2 inv = make_float2(p.inv_scale, p.inv_scale);
  int si = 0, hop = 1;
  if ((int)blockIdx.x < p.n_tiles) si = find_seg(p, blockIdx.x);
  for (int t = blockIdx.x; t < p.n_tiles; t += gridDim.x) {
    si = next_seg(p, si, t, hop);
    const NormSeg& sg = p.seg[si];
    if (!DOPT_TILE_OK(p, kSiteListNorm, (int64_t)(t - sg.tile0) * (kNormTileBytes / (sg.dtype == DOPT_F32 ? 4 : 2)), 1,
                      sg.len + sg.shift))
      continue;
    if (sg.dtype == DOPT_F32)
      norm_tile<float>(sg, t, inv, acc);
    else if (sg.dtype == DOPT_BF16)
      norm_tile<__nv_bfloat16>(sg, t, inv, acc);
    else
      norm_tile<__half>(sg, t, inv, acc);
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
    if (blockIdx.x == 0) *p.err_flag = 0;
    p.partials[blockIdx.x] = Partial{s_sum[0], isfinite(s_sum[0]) ? 0 : 1, s_zero[0]};
  }
}

// The finalize of a call: one CTA, launched to start under the last norm
// launch and waiting for it (and so for the ones before it, which that one
// waited for) before it reads their partials.  128 threads: up to 608 slots
// are one round of loads, and fewer warps share the SM's slow fp64 unit (256:
// 2 to 4 % on small lists, 512: 12 %).
constexpr int kFinalizeThreads = 128;
__global__ void __launch_bounds__(kFinalizeThreads) tensors_finalize(const __grid_constant__ FinalizeParams p) {
  allow_dependent_launch();  // the AdamW launch behind it waits for this grid
  wait_for_prior_grids();
  finalize_block<kFinalizeThreads>(p.fin);
}

int tensors_norm_tile_bytes() { return kNormTileBytes; }

int tensors_norm_grid(const NormParamsT<kNormCap>& p, int* grid) {
  const char* what = "tensors_norm launch";
  int st = p.n_seg <= kNormSmallCap ? resident_ctas<tensors_norm<kNormSmallCap>>(grid, what)
                                    : resident_ctas<tensors_norm<kNormCap>>(grid, what);
  *grid = std::max(1, std::min(*grid, p.n_tiles));
  return st;
}

int launch_tensors_norm(const NormParamsT<kNormCap>& p, cudaStream_t s) {
  const char* what = "tensors_norm launch";
  if (p.n_seg <= kNormSmallCap)
    return launch_table<tensors_norm<kNormSmallCap>>(compact_table<NormParamsT<kNormSmallCap>, NormHead>(p), s, what);
  return launch_table<tensors_norm<kNormCap>>(p, s, what);
}

int launch_tensors_finalize(const FinalizeArgs& fin, cudaStream_t s) {
  return launch_table<tensors_finalize, 0, kFinalizeThreads>(FinalizeParams{fin, 1}, s, "tensors_finalize launch", true);
}

}  // namespace dopt
