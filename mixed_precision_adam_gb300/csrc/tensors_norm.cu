// tensors_norm.cu -- the grad norm over a list of tensors: one pass over the
// grads, sum of squares, non-finite flag and zero count per CTA, and the
// finalize (norm, clip coefficient, skip decision) in the last CTA.
#include "tensors.cuh"

namespace dopt {

// Squares of a chunk whose fp32 sum would over- or underflow, in fp64.
static __device__ __noinline__ double chunk_wide(const float* x, int n) {
  double d = 0.0;
  for (int j = 0; j < n; ++j) d += (double)x[j] * (double)x[j];
  return d;
}

template <typename GT>
__device__ __forceinline__ void norm_tile(const NormSeg& sg, int64_t off, int n, float inv, double& sum, int& zeros) {
  const GT* g = static_cast<const GT*>(sg.grad) + off;
  for (int e = threadIdx.x; e < n; e += kThreads) {
    const float x = __fmul_rn(widen<GT>(g[e]), inv);
    zeros += x == 0.f;
    const float sq = __fmul_rn(x, x);
    sum += (sq <= 0x1p100f && sq >= 0x1p-90f) ? (double)sq : chunk_wide(&x, 1);
  }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) tensors_norm(const __grid_constant__ NormParamsT<CAP> p) {
  double sum = 0.0;
  int zeros = 0;
  int si = 0;
  if ((int)blockIdx.x < p.n_tiles) si = find_seg(p, blockIdx.x);
  for (int t = blockIdx.x; t < p.n_tiles; t += gridDim.x) {
    si = next_seg(p, si, t);
    const NormSeg& sg = p.seg[si];
    const int64_t off = (int64_t)(t - sg.tile0) * kNormTile;
    const int n = (int)min((int64_t)kNormTile, sg.len - off);
    if (sg.dtype == DOPT_F32)
      norm_tile<float>(sg, off, n, p.inv_scale, sum, zeros);
    else if (sg.dtype == DOPT_BF16)
      norm_tile<__nv_bfloat16>(sg, off, n, p.inv_scale, sum, zeros);
    else
      norm_tile<__half>(sg, off, n, p.inv_scale, sum, zeros);
  }
  allow_dependent_launch();
  __shared__ double s_sum[kThreads / 32];
  __shared__ int s_zero[kThreads / 32];
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
