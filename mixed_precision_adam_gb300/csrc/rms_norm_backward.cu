// rms_norm_backward.cu -- the backward pass of the RMS norm.
//
// A CTA adds up its rows' dy * hat in registers, a column always in the same
// thread; the CTAs' sums are added by a launch of its own in a fixed order.
#include "rms_norm.cuh"

namespace dopt {

// Rows' values under way under the row before's work, where there is room.
template <typename T, int V>
constexpr bool kBackAhead = V * sizeof(T) <= 4;

template <typename T, int G, int V, bool VEC>
__global__ void __launch_bounds__(kRowThreads<G>) rms_norm_backward(const __grid_constant__ NormBackRows p) {
  __shared__ float s_sum[2][32];
  __shared__ float s_gain[G == 32 ? 8 * 32 * 8 : 1];
  using Piece = Eight8<T, VEC>;
  const int g = threadIdx.x % G;
  const uint32_t key = drop_key(p.drop);
  const T* h = static_cast<const T*>(p.h.data);
  const T* dy = static_cast<const T*>(p.dy.data);
  const T* dres = static_cast<const T*>(p.dres.data);
  const int64_t stride = (int64_t)gridDim.x * kRowsAtOnce<G>;
  int64_t row = (int64_t)blockIdx.x * kRowsAtOnce<G> + threadIdx.x / G;
  Piece hs[V], ys[V], rs[V];
  float rstd = 0.f;
  auto load = [&](int64_t at) {
    rstd = p.rstd[at];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = first_column<V, VEC, G>(g, v);
      hs[v].load(h + at * p.h.ld + c, p.cols - c);
      ys[v].load(dy + at * p.dy.ld + c, p.cols - c);
      if (dres) rs[v].load(dres + at * p.dres.ld + c, p.cols - c);
    }
  };
  if (row < p.rows) load(row);
  float gain[V][8], acc[V][8];
  load_gain<T, V, VEC, G>(p.gain, p.gain_f32, g, p.cols, gain);
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[v][j] = 0.f;
  int turn = 0;
  for (; row < p.rows; row += stride) {
    float hat[V][8], d[V][8], dot = 0.f;
    const float r0 = rstd;
    Piece res[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      hs[v].widen8(hat[v]);
      ys[v].widen8(d[v]);
      if (dres) res[v] = rs[v];
    }
    if (kBackAhead<T, V> && row + stride < p.rows) load(row + stride);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        hat[v][j] *= r0;
        acc[v][j] = fmaf(d[v][j], hat[v][j], acc[v][j]);
        d[v][j] *= gain[v][j];
        dot = fmaf(d[v][j], hat[v][j], dot);
      }
    dot = row_sum<G>(dot, s_sum[turn]) / (float)p.cols;
    turn ^= 1;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = first_column<V, VEC, G>(g, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) d[v][j] = r0 * fmaf(-hat[v][j], dot, d[v][j]);
      if (dres) {
        float r[8];
        res[v].widen8(r);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[v][j] += r[j];
      }
      if (p.dh.data) Piece::store(static_cast<T*>(p.dh.data) + row * p.dh.ld + c, p.cols - c, d[v]);
      if (p.dx.data) {
        drop_eight<VEC>(d[v], (uint64_t)row * p.cols + c, p.drop, key);
        Piece::store(static_cast<T*>(p.dx.data) + row * p.dx.ld + c, p.cols - c, d[v]);
      }
    }
    if (!kBackAhead<T, V> && row + stride < p.rows) load(row + stride);
  }
  allow_dependent_launch();
  if (!p.partial) return;
  float* part = p.partial + (int64_t)blockIdx.x * p.cols;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = first_column<V, VEC, G>(g, v);
    if constexpr (G == 32) {
      // the warps' sums of these columns, in the warps' order
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) s_gain[(threadIdx.x / 32 * 8 + j) * 32 + g] = acc[v][j];
      __syncthreads();
      const int j = threadIdx.x / 32, at = c + j * kColumnStep<VEC>;
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) sum += s_gain[(w * 8 + j) * 32 + g];
      if (at < p.cols) part[at] = sum;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = c + j * kColumnStep<VEC>;
        if (at < p.cols) part[at] = acc[v][j];
      }
    }
  }
}

struct GainParams {
  const float* partial;
  float* dgain;
  int32_t parts, cols, accumulate;
  int32_t n_tiles;
};
constexpr int kGainColumns = 32, kGainThreads = 1024;
// 32 columns per CTA, each warp a share of the partial sums, eight loads at a
// time.  Started under the kernel before it.
__global__ void __launch_bounds__(kGainThreads) rms_norm_gain(const __grid_constant__ GainParams p) {
  __shared__ float s_sum[kGainThreads / 32][33];
  constexpr int kWarps = kGainThreads / 32, kAhead = 8;
  const int lane = threadIdx.x % 32, c = blockIdx.x * kGainColumns + lane, w = threadIdx.x / 32;
  wait_for_prior_grids();
  float sum = 0.f;
  if (c < p.cols)
    for (int k = w; k < p.parts; k += kWarps * kAhead) {
      float t[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) t[j] = k + j * kWarps < p.parts ? p.partial[(int64_t)(k + j * kWarps) * p.cols + c] : 0.f;
#pragma unroll
      for (int j = 0; j < kAhead; ++j) sum += t[j];
    }
  s_sum[w][lane] = sum;
  __syncthreads();
  // a warp adds the warps' sums of a column, in a fixed order
  float x = s_sum[lane][w];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  const int at = blockIdx.x * kGainColumns + w;
  if (lane == 0 && at < p.cols) p.dgain[at] = p.accumulate ? p.dgain[at] + x : x;
}

namespace {

// Each CTA should have rows enough that its partial sums are a small part of
// what it reads.
constexpr int kRowsPerPart = 8;

template <typename T, int G, int V, bool VEC>
int launch_one(const NormBackRows& p, cudaStream_t s, int* parts) {
  const char* what = "rms_norm_backward launch";
  const int64_t rows = kRowsAtOnce<G> > kRowsPerPart || !p.partial ? kRowsAtOnce<G> : kRowsPerPart;
  int grid = 0;
  if (int st = row_grid<rms_norm_backward<T, G, V, VEC>, kRowThreads<G>>(
          p, std::min<int64_t>(kMaxParts, (p.rows + rows - 1) / rows), &grid, what))
    return st;
  *parts = grid;
  return launch_table<rms_norm_backward<T, G, V, VEC>, 0, kRowThreads<G>>(p, s, what, false, grid);
}
template <typename T, bool VEC>
int launch_length(const NormBackRows& p, cudaStream_t s, int* parts) {
  const int c = p.cols;
  if (c <= 256) return launch_one<T, 32, 1, VEC>(p, s, parts);
  if (c <= 512) return launch_one<T, 32, 2, VEC>(p, s, parts);
  if (c <= 1024) return launch_one<T, 128, 1, VEC>(p, s, parts);
  if (c <= 2048) return launch_one<T, 256, 1, VEC>(p, s, parts);
  if (c <= 4096) return launch_one<T, 256, 2, VEC>(p, s, parts);
  if (c <= 8192) return launch_one<T, 512, 2, VEC>(p, s, parts);
  return launch_one<T, 512, 4, VEC>(p, s, parts);
}

}  // namespace

int launch_norm_backward(int32_t dtype, bool vec, const NormBackRows& p, cudaStream_t s, int* parts) {
  if (dtype == DOPT_F32) return vec ? launch_length<float, true>(p, s, parts) : launch_length<float, false>(p, s, parts);
  if (dtype == DOPT_BF16)
    return vec ? launch_length<__nv_bfloat16, true>(p, s, parts) : launch_length<__nv_bfloat16, false>(p, s, parts);
  return vec ? launch_length<__half, true>(p, s, parts) : launch_length<__half, false>(p, s, parts);
}

int launch_norm_gain(const float* partial, int parts, int32_t cols, float* dgain, bool accumulate, cudaStream_t s) {
  GainParams g{partial, dgain, parts, cols, accumulate ? 1 : 0, (cols + kGainColumns - 1) / kGainColumns};
  return launch_table<rms_norm_gain, 0, kGainThreads>(g, s, "rms_norm_gain launch", true, g.n_tiles);
}

}  // namespace dopt
