// rms_norm_backward.cu -- the backward pass of the RMS norm.
//
// A CTA adds up its rows' dy * hat in registers, a column always in the same
// thread; the CTAs' sums are added by a launch of its own in a fixed order.
// 32768 x 4096 bf16 with dres: 174 us, 6.2 TB/s of 8 bytes per element.
#include "rms_norm.cuh"

namespace dopt {

// Rows' values under way under the row before's work, where there is room.
template <typename T, int V>
constexpr bool kBackAhead = V * sizeof(T) <= 4;

// Threads and CTAs per SM that a kernel is compiled for: short rows of 16-bit
// values in 80 registers, for three CTAs (2048 columns: 75 us against 85 with
// one register more).
template <typename T, int V, bool VEC, int WARPS>
constexpr bool kShortRows = V == 1 && VEC && sizeof(T) == 2 && WARPS > 0;
template <typename T, int V, bool VEC, int WARPS>
constexpr int kRowBound = WARPS == 0 || kShortRows<T, V, VEC, WARPS> ? 256 : kMaxRowThreads;
template <typename T, int V, bool VEC, int WARPS>
constexpr int kRowCtas = V == 1 && VEC && sizeof(T) == 2 ? 3 : WARPS > 0 ? 1 : V == 1 || VEC ? 2 : 1;

template <typename T, int V, bool VEC, int WARPS>
__global__ void __launch_bounds__(kRowBound<T, V, VEC, WARPS>, kRowCtas<T, V, VEC, WARPS>) rms_norm_backward(const __grid_constant__ NormBackRows p) {
  constexpr bool WARP = kWarpRows<WARPS>;
  __shared__ RowSums s_sum[2];
  __shared__ float s_gain[WARP ? 8 * 32 * 8 : 1];
  using Piece = Eight8<T, VEC>;
  const RowShape<WARP> at;
  clear_sums<WARPS>(s_sum);
  const uint32_t key = drop_key(p.drop);
  const T* h = static_cast<const T*>(p.h.data);
  const T* dy = static_cast<const T*>(p.dy.data);
  const T* dres = static_cast<const T*>(p.dres.data);
  const int64_t stride = at.stride();
  int64_t row = at.first();
  Piece hs[V], ys[V], rs[V];
  float rstd = 0.f;
  auto load = [&](int64_t r) {
    rstd = p.rstd[r];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = at.template column<V, VEC>(v);
      hs[v].load(h + r * p.h.ld + c, p.cols - c);
      ys[v].load(dy + r * p.dy.ld + c, p.cols - c);
      if (dres && kBackAhead<T, V>) rs[v].load(dres + r * p.dres.ld + c, p.cols - c);
    }
  };
  if (row < p.rows) load(row);
  const RowGain<T, V, VEC, WARP, V <= 2> gain(p.gain, p.gain_f32, at, p.cols);
  float2 acc[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[v][k] = make_float2(0.f, 0.f);
  int turn = 0;
  for (; row < p.rows; row += stride) {
    float2 hat[V][4], d[V][4], dots = make_float2(0.f, 0.f);
    const float r0 = rstd;
    Piece res[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      hs[v].widen8(hat[v]);
      ys[v].widen8(d[v]);
      if (dres && kBackAhead<T, V>) res[v] = rs[v];
    }
    if (kBackAhead<T, V> && row + stride < p.rows) load(row + stride);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float2 w[4];
      gain.of(at, v, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        hat[v][k] = __fmul2_rn(hat[v][k], both_of(r0));
        acc[v][k] = __ffma2_rn(d[v][k], hat[v][k], acc[v][k]);
        d[v][k] = __fmul2_rn(d[v][k], w[k]);
        dots = __ffma2_rn(d[v][k], hat[v][k], dots);
      }
    }
    const float mean = row_sum<WARPS>(dots.x + dots.y, s_sum[turn]) / (float)p.cols;
    turn ^= 1;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = at.template column<V, VEC>(v);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        d[v][k] = __fmul2_rn(__ffma2_rn(hat[v][k], both_of(-mean), d[v][k]), both_of(r0));
      if (dres) {
        float2 r[4];
        if (!kBackAhead<T, V>) res[v].load(dres + row * p.dres.ld + c, p.cols - c);
        res[v].widen8(r);
#pragma unroll
        for (int k = 0; k < 4; ++k) d[v][k] = __fadd2_rn(d[v][k], r[k]);
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
    const int c = at.template column<V, VEC>(v);
    if constexpr (WARP) {
      // the warps' sums of these columns, in the warps' order
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) s_gain[(threadIdx.x / 32 * 8 + j) * 32 + at.g] = j & 1 ? acc[v][j / 2].y : acc[v][j / 2].x;
      __syncthreads();
      const int j = threadIdx.x / 32, col = c + j * kColumnStep<VEC>;
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) sum += s_gain[(w * 8 + j) * 32 + at.g];
      if (col < p.cols) part[col] = sum;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int col = c + j * kColumnStep<VEC>;
        if (col < p.cols) part[col] = j & 1 ? acc[v][j / 2].y : acc[v][j / 2].x;
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

// CTAs that a call asks for.  Without dgain each row may have one.  With it
// each has eight rows, and 32 where there are more than 608 such, so that its
// partial sums are a small part of what it reads and that adding them takes
// little time; but as many as the device has SMs, rows allowing: 8, 64 and 608
// rows of 4096 bf16 columns take 5.7, 7.1 and 10.2 us so, 10.2, 10.3 and 11.8
// with eight rows for each CTA (2.3, 2.3 and 3.9 without dgain).
int64_t parts_asked(const NormBackRows& p, int rows_at_once, int sms) {
  const int64_t all = (p.rows + rows_at_once - 1) / rows_at_once;
  if (!p.partial) return std::min<int64_t>(all, max_parts(p.cols));
  const int64_t few = std::min<int64_t>({all, std::max<int64_t>(sms, (p.rows + 7) / 8), 608});
  return std::min<int64_t>({all, std::max<int64_t>(few, p.rows / 32), max_parts(p.cols)});
}

template <typename T, int V, bool VEC, int WARPS>
int launch_one(const NormBackRows& p, cudaStream_t s, int* parts) {
  const char* what = "rms_norm_backward launch";
  constexpr int kRows = RowShape<kWarpRows<WARPS>>::kAtOnce;
  const int threads = row_threads<V, kWarpRows<WARPS>>(p.cols);
  int sms = 0;
  if (int st = device_sms(&sms)) return st;
  if (int st = row_grid<rms_norm_backward<T, V, VEC, WARPS>>(threads, parts_asked(p, kRows, sms), parts, what)) return st;
  return launch_row_kernel<rms_norm_backward<T, V, VEC, WARPS>>(p, *parts, threads, s, what);
}
template <typename T, bool VEC>
int launch_length(const NormBackRows& p, cudaStream_t s, int* parts) {
  const int c = p.cols;
  if (c <= 256) return launch_one<T, 1, VEC, 0>(p, s, parts);
  if (c <= 512) return launch_one<T, 2, VEC, 0>(p, s, parts);
  if (c <= 2048) return launch_one<T, 1, VEC, 8>(p, s, parts);
  if (c <= 4096) {
    if constexpr (sizeof(T) == 2)
      return launch_one<T, 2, VEC, 8>(p, s, parts);
    else
      return launch_one<T, 1, VEC, 16>(p, s, parts);
  }
  if (c <= 8192) return launch_one<T, 2, VEC, 16>(p, s, parts);
  return launch_one<T, 4, VEC, 16>(p, s, parts);
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
