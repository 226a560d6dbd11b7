// rms_norm.cuh -- what the RMS norm and its backward pass share: rows spread
// over threads, sums over a row, and the choice of a kernel by row length.
//
// Both are bound by memory: each value is read once and stays in registers
// between the row's sum and its use, and a row's loads are under way while
// the row before is worked on.  A warp has a row that fits it, so that its
// sum needs no shared memory; longer ones have just the warps that they fill,
// each thread V times eight columns: lanes without columns issue all the same.
#pragma once

#include "matrix8.cuh"

namespace dopt {

struct RowsIn {
  const void* data;
  int64_t ld;
};
struct RowsOut {
  void* data;
  int64_t ld;
};

// Rows spread over threads.  WARP: a warp has a row, a CTA eight rows; else
// a CTA has one, of as many warps as its length asks for.
template <bool WARP>
struct RowShape {
  static constexpr int kAtOnce = WARP ? 8 : 1;
  int g, threads;  // this thread's place in its row, and the row's threads
  __device__ __forceinline__ RowShape()
      : g(WARP ? threadIdx.x % 32 : threadIdx.x), threads(WARP ? 32 : blockDim.x) {}
  __device__ __forceinline__ int64_t first() const { return (int64_t)blockIdx.x * kAtOnce + (WARP ? threadIdx.x / 32 : 0); }
  __device__ __forceinline__ int64_t stride() const { return (int64_t)gridDim.x * kAtOnce; }
  // First of the thread's eight columns in its v-th piece of V: consecutive
  // ones (VEC), or 32 apart in its warp's part of the row.
  template <int V, bool VEC>
  __device__ __forceinline__ int column(int v) const {
    return VEC ? (v * threads + g) * 8 : (g / 32) * (256 * V) + v * 256 + g % 32;
  }
};
template <bool VEC>
constexpr int kColumnStep = VEC ? 1 : 32;
constexpr int kMaxRowThreads = 512;

// Rows of at most WARPS warps each, 0: a warp has a row (WARP above).
template <int WARPS>
constexpr bool kWarpRows = WARPS == 0;

// A sum over the threads that have a row.  The warps' sums lie in shared
// memory, zeros for the warps that a CTA does not have, so that all of them
// are read at once (a loop over the warps took a row 30 cycles for each).
struct RowSums {
  float of_warp[kMaxRowThreads / 32];
};
template <int WARPS>
__device__ __forceinline__ void clear_sums(RowSums (&s)[2]) {
  if constexpr (WARPS > 0) {
    if (threadIdx.x < kMaxRowThreads / 32) s[0].of_warp[threadIdx.x] = s[1].of_warp[threadIdx.x] = 0.f;
    __syncthreads();
  }
}
template <int WARPS>
__device__ __forceinline__ float row_sum(float x, RowSums& s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  if constexpr (WARPS > 0) {
    if (threadIdx.x % 32 == 0) s.of_warp[threadIdx.x / 32] = x;
    __syncthreads();
    x = s.of_warp[0];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) x += s.of_warp[w];
  }
  return x;
}

// A thread's values of the gain, zeros past the end: kept in registers, or
// read again for each row where those are short.
template <typename T, int V, bool VEC, bool WARP, bool KEPT>
struct RowGain {
  static constexpr bool kKept = KEPT;
  const void* gain;
  bool f32;
  int cols;
  float2 kept[kKept ? V : 1][4];
  __device__ __forceinline__ RowGain(const void* gain_, bool f32_, const RowShape<WARP>& at, int cols_)
      : gain(gain_), f32(f32_), cols(cols_) {
    if constexpr (kKept)
#pragma unroll
      for (int v = 0; v < V; ++v) read(at, v, kept[v]);
  }
  __device__ __forceinline__ void read(const RowShape<WARP>& at, int v, float2 (&out)[4]) const {
    if constexpr (VEC) {
      const int c = at.template column<V, VEC>(v);
      if (f32) {
        Eight8<float, true> r;
        r.load(static_cast<const float*>(gain) + c, cols - c);
        r.widen8(out);
      } else {
        Eight8<T, true> r;
        r.load(static_cast<const T*>(gain) + c, cols - c);
        r.widen8(out);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = at.template column<V, VEC>(v) + 64 * k;
        out[k] = make_float2(one(c), one(c + 32));
      }
    }
  }
  __device__ __forceinline__ float one(int c) const {
    return c < cols ? (f32 ? __ldg(static_cast<const float*>(gain) + c) : widen<T>(static_cast<const T*>(gain)[c])) : 0.f;
  }
  __device__ __forceinline__ void of(const RowShape<WARP>& at, int v, float2 (&out)[4]) const {
    if constexpr (kKept) {
#pragma unroll
      for (int k = 0; k < 4; ++k) out[k] = kept[v][k];
    } else {
      read(at, v, out);
    }
  }
};

// Threads of a CTA for rows of this length.
template <int V, bool WARP>
int row_threads(int32_t cols) {
  return WARP ? 256 : (cols + 256 * V - 1) / (256 * V) * 32;
}

// As many CTAs as the device holds at once, at most `most`.
template <auto Kern>
int row_grid(int threads, int64_t most, int* grid, const char* what) {
  static std::atomic<int> known[64][kMaxRowThreads / 32 + 1];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(DOPT_E_CUDA, std::string("cudaGetDevice: ") + cudaGetErrorString(e));
  int ctas = dev < 64 ? known[dev][threads / 32].load(std::memory_order_relaxed) : 0;
  if (!ctas) {
    int sms = 0, per_sm = 0;
    if (int st = device_sms(&sms)) return st;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, Kern, threads, 0);
    if (e != cudaSuccess || per_sm < 1)
      return fail(DOPT_E_CUDA, std::string(what) + ": occupancy query: " + cudaGetErrorString(e));
    ctas = per_sm * sms;
    if (dev < 64) known[dev][threads / 32].store(ctas, std::memory_order_relaxed);
  }
  *grid = (int)std::max<int64_t>(1, std::min<int64_t>(ctas, most));
  return DOPT_OK;
}
// Launch of a kernel over rows, with a CTA size known at run time.
template <auto Kern, typename P>
int launch_row_kernel(const P& params, int grid, int threads, cudaStream_t s, const char* what) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = s;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, Kern, params);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(DOPT_E_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
  }
  return check_launch(what);
}

// ----------------------------------------------------------- backward pass --

struct NormBackRows {
  RowsIn dy, h, dres;
  RowsOut dh, dx;
  const void* gain;
  const float* rstd;
  float* partial;  // of dgain, a row of cols per CTA; or NULL
  int64_t rows;
  int32_t cols;
  Drop drop;
  bool gain_f32;
};
// CTAs of the backward pass, and so partial sums: as many as 12 per SM of 152
// where rows are short and CTAs small.
__host__ __device__ constexpr int max_parts(int64_t cols) { return cols <= 2048 ? 1824 : 608; }

// See rms_norm_backward.cu; *parts receives the number of partial sums.
int launch_norm_backward(int32_t dtype, bool vec, const NormBackRows& p, cudaStream_t s, int* parts);
int launch_norm_gain(const float* partial, int parts, int32_t cols, float* dgain, bool accumulate, cudaStream_t s);

}  // namespace dopt
