// rms_norm.cuh -- what the RMS norm and its backward pass share: rows spread
// over threads, sums over a row, and the choice of a kernel by row length.
//
// Both are bound by memory: each value is read once and stays in registers
// between the row's sum and its use, and a row's loads are under way while
// the row before is worked on.  G threads have a row, each of them V times
// eight columns; a warp where a row fits it, so that its sum needs no shared
// memory.
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

// Rows that a CTA has at once, and its threads.
template <int G>
constexpr int kRowsAtOnce = G == 32 ? 8 : 1;
template <int G>
constexpr int kRowThreads = G == 32 ? 256 : G;

// First of a thread's eight columns in its v-th piece: consecutive ones
// (VEC), or 32 apart in its warp's part of the row.
template <int V, bool VEC, int G>
__device__ __forceinline__ int first_column(int g, int v) {
  return VEC ? (v * G + g) * 8 : (g / 32) * (256 * V) + v * 256 + g % 32;
}
template <bool VEC>
constexpr int kColumnStep = VEC ? 1 : 32;

// A sum over the G threads that have a row.
template <int G>
__device__ __forceinline__ float row_sum(float x, float (&s_sum)[32]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  if constexpr (G > 32) {
    if (threadIdx.x % 32 == 0) s_sum[threadIdx.x / 32] = x;
    __syncthreads();
    x = s_sum[0];
#pragma unroll
    for (int w = 1; w < G / 32; ++w) x += s_sum[w];
  }
  return x;
}

// A thread's values of the gain, zeros past the end.
template <typename T, int V, bool VEC, int G>
__device__ __forceinline__ void load_gain(const void* gain, bool f32, int g, int cols, float (&out)[V][8]) {
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int at = first_column<V, VEC, G>(g, v) + j * kColumnStep<VEC>;
      out[v][j] = at < cols ? (f32 ? __ldg(static_cast<const float*>(gain) + at) : widen<T>(static_cast<const T*>(gain)[at])) : 0.f;
    }
}

// As many CTAs as the device holds at once and the rows ask for.
template <auto Kern, int THREADS, typename P>
int row_grid(const P& p, int64_t ctas_asked, int* grid, const char* what) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(DOPT_E_CUDA, std::string("cudaGetDevice: ") + cudaGetErrorString(e));
  int ctas = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (!ctas) {
    int sms = 0, per_sm = 0;
    if (int st = device_sms(&sms)) return st;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, Kern, THREADS, 0);
    if (e != cudaSuccess || per_sm < 1)
      return fail(DOPT_E_CUDA, std::string(what) + ": occupancy query: " + cudaGetErrorString(e));
    ctas = per_sm * sms;
    if (dev < 64) known[dev].store(ctas, std::memory_order_relaxed);
  }
  *grid = (int)std::max<int64_t>(1, std::min<int64_t>(ctas, ctas_asked));
  return DOPT_OK;
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
  int32_t n_tiles;
};
constexpr int kMaxParts = 608;  // CTAs of the backward pass, at most

// See rms_norm_backward.cu; *parts receives the number of partial sums.
int launch_norm_backward(int32_t dtype, bool vec, const NormBackRows& p, cudaStream_t s, int* parts);
int launch_norm_gain(const float* partial, int parts, int32_t cols, float* dgain, bool accumulate, cudaStream_t s);

}  // namespace dopt
