// rms_norm.cu -- the RMS norm with the residual's addition, values or 8-bit
// codes out, and its backward pass.
//
// Both are bound by memory: each value is read once and stays in registers
// between the row's sum and its use.  G threads have a row, each of them V
// vectors of eight consecutive columns; a warp where a row fits it, so that
// its sum needs no shared memory.
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

struct NormRows {
  RowsIn x, residual;
  RowsOut h, y;
  const void* gain;
  uint8_t* codes;
  uint8_t* scales;
  int64_t ld_codes;
  float* rstd;
  int64_t rows;
  int32_t cols;
  uint32_t groups;  // of scale bytes
  float eps;
  Drop drop;
  bool vec, gain_f32;
  int32_t n_tiles;  // groups of threads' rows, for the launch
};

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
template <int G>
__device__ __noinline__ double row_sum_wide(double x, double (&s_sum)[32]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  if constexpr (G > 32) {
    if (threadIdx.x % 32 == 0) s_sum[threadIdx.x / 32] = x;
    __syncthreads();
    x = s_sum[0];
    for (int w = 1; w < G / 32; ++w) x += s_sum[w];
    __syncthreads();
  }
  return x;
}

// A gain's eight values from column c on, zeros past the end.
template <typename T>
__device__ __forceinline__ void load_gain(const void* gain, bool f32, int c, int cols, float (&g)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int at = c + j;
    g[j] = at < cols ? (f32 ? __ldg(static_cast<const float*>(gain) + at) : widen<T>(static_cast<const T*>(gain)[at])) : 0.f;
  }
}

// Rows that a CTA has at once, and its threads.
template <int G>
constexpr int kRowsAtOnce = G == 32 ? 8 : 1;
template <int G>
constexpr int kRowThreads = G == 32 ? 256 : G;

template <typename T, int G, int V>
__global__ void __launch_bounds__(kRowThreads<G>) rms_norm(const __grid_constant__ NormRows p) {
  __shared__ float s_sum[2][32];
  __shared__ double s_wide[32];
  const int g = threadIdx.x % G;
  const uint32_t key = drop_key(p.drop);
  float gain[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) load_gain<T>(p.gain, p.gain_f32, (v * G + g) * 8, p.cols, gain[v]);
  const int64_t stride = (int64_t)gridDim.x * kRowsAtOnce<G>;
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * kRowsAtOnce<G> + threadIdx.x / G; row < p.rows; row += stride) {
    float f[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * G + g) * 8, n = max(0, min(8, p.cols - c));
      load_some(static_cast<const T*>(p.x.data) + row * p.x.ld + c, n, p.vec, f[v]);
    }
    if (p.residual.data || p.drop.threshold) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = (v * G + g) * 8, n = max(0, min(8, p.cols - c));
        if (p.drop.threshold && n > 0) drop_eight(f[v], (uint64_t)row * p.cols + c, p.drop, key);
        if (p.residual.data) {
          float r[8];
          load_some(static_cast<const T*>(p.residual.data) + row * p.residual.ld + c, n, p.vec, r);
#pragma unroll
          for (int j = 0; j < 8; ++j) f[v][j] += r[j];
        }
        // what the norm sees is what is stored: the backward pass, and a
        // norm of h alone, then see the same
#pragma unroll
        for (int j = 0; j < 8; ++j) f[v][j] = j < n ? widen<T>(narrow<T>(f[v][j])) : 0.f;
        if (p.h.data) store_some(static_cast<T*>(p.h.data) + row * p.h.ld + c, n, p.vec, f[v]);
      }
    }
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(f[v][j], f[v][j], sum);
    sum = row_sum<G>(sum, s_sum[turn]);
    turn ^= 1;
    float rstd;
    if (isfinite(sum)) {
      const float m = sum / (float)p.cols + p.eps;
      rstd = rsqrtf(m);
      // one step of Newton's method, as rsqrtf may be two last places off
      if (m > 1e-30f) rstd *= fmaf(-0.5f * m * rstd, rstd, 1.5f);
    } else {
      double wide = 0.0;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int j = 0; j < 8; ++j) wide += (double)f[v][j] * (double)f[v][j];
      wide = row_sum_wide<G>(wide, s_wide);
      rstd = (float)(1.0 / sqrt(wide / (double)p.cols + (double)p.eps));
    }
    if (g == 0 && p.rstd) p.rstd[row] = rstd;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * G + g) * 8, n = max(0, min(8, p.cols - c));
#pragma unroll
      for (int j = 0; j < 8; ++j) f[v][j] = j < n ? f[v][j] * rstd * gain[v][j] : 0.f;
      if (p.y.data) store_some(static_cast<T*>(p.y.data) + row * p.y.ld + c, n, p.vec, f[v]);
      if (p.codes) {
        // a block of 128 columns is sixteen threads'
        uint32_t top = top_of(f[v]);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        const uint32_t s = m_scale_of(top);
        const float up = code_factor(s);
        const uint2 code = make_uint2(four_codes(f[v], up, s == 255u), four_codes(f[v] + 4, up, s == 255u));
        uint8_t* dst = p.codes + row * p.ld_codes + c;
        if (n == 8) {
          *reinterpret_cast<uint2*>(dst) = code;
        } else {
          for (int j = 0; j < n; ++j) dst[j] = (uint8_t)((j < 4 ? code.x : code.y) >> (8 * (j & 3)));
        }
        if (g % 16 == 0 && n > 0) p.scales[scale_place(row, c / kBlock8, p.groups)] = (uint8_t)s;
      }
    }
  }
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
  bool vec, gain_f32;
  int32_t n_tiles;
};

// A CTA adds up its rows' dy * hat in registers, a column always in the same
// thread; the CTAs' sums are added by a launch of its own in a fixed order.
constexpr int kMaxParts = 608;  // CTAs, at most

template <typename T, int G, int V>
__global__ void __launch_bounds__(kRowThreads<G>) rms_norm_backward(const __grid_constant__ NormBackRows p) {
  __shared__ float s_sum[2][32];
  __shared__ float s_gain[G == 32 ? 8 * 32 * 8 : 1];
  const int g = threadIdx.x % G;
  const uint32_t key = drop_key(p.drop);
  float gain[V][8], acc[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    load_gain<T>(p.gain, p.gain_f32, (v * G + g) * 8, p.cols, gain[v]);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[v][j] = 0.f;
  }
  const int64_t stride = (int64_t)gridDim.x * kRowsAtOnce<G>;
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * kRowsAtOnce<G> + threadIdx.x / G; row < p.rows; row += stride) {
    const float rstd = p.rstd[row];
    float hat[V][8], dy[V][8], dot = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * G + g) * 8, n = max(0, min(8, p.cols - c));
      load_some(static_cast<const T*>(p.h.data) + row * p.h.ld + c, n, p.vec, hat[v]);
      load_some(static_cast<const T*>(p.dy.data) + row * p.dy.ld + c, n, p.vec, dy[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        hat[v][j] *= rstd;
        acc[v][j] = fmaf(dy[v][j], hat[v][j], acc[v][j]);
        dy[v][j] *= gain[v][j];
        dot = fmaf(dy[v][j], hat[v][j], dot);
      }
    dot = row_sum<G>(dot, s_sum[turn]) / (float)p.cols;
    turn ^= 1;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = (v * G + g) * 8, n = max(0, min(8, p.cols - c));
      if (n == 0) continue;
      float r[8];
      if (p.dres.data) load_some(static_cast<const T*>(p.dres.data) + row * p.dres.ld + c, n, p.vec, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dy[v][j] = rstd * fmaf(-hat[v][j], dot, dy[v][j]);
        if (p.dres.data) dy[v][j] += r[j];
      }
      if (p.dh.data) store_some(static_cast<T*>(p.dh.data) + row * p.dh.ld + c, n, p.vec, dy[v]);
      if (p.dx.data) {
        drop_eight(dy[v], (uint64_t)row * p.cols + c, p.drop, key);
        store_some(static_cast<T*>(p.dx.data) + row * p.dx.ld + c, n, p.vec, dy[v]);
      }
    }
  }
  if (!p.partial) return;
  float* part = p.partial + (int64_t)blockIdx.x * p.cols;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = (v * G + g) * 8;
    if constexpr (G == 32) {
      // the warps' sums of these columns, in the warps' order
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) s_gain[(threadIdx.x / 32 * 8 + j) * 32 + g] = acc[v][j];
      __syncthreads();
      const int j = threadIdx.x / 32;
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) sum += s_gain[(w * 8 + j) * 32 + g];
      if (c + j < p.cols) part[c + j] = sum;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < p.cols) part[c + j] = acc[v][j];
    }
  }
}

struct GainParams {
  const float* partial;
  float* dgain;
  int32_t parts, cols, accumulate;
  int32_t n_tiles;
};
constexpr int kGainColumns = 32;
// 32 columns per CTA, each warp a share of the partial sums.
__global__ void __launch_bounds__(kThreads) rms_norm_gain(const __grid_constant__ GainParams p) {
  __shared__ float s_sum[kThreads / 32][32];
  const int c = blockIdx.x * kGainColumns + threadIdx.x % 32, w = threadIdx.x / 32;
  float sum = 0.f;
  if (c < p.cols)
    for (int k = w; k < p.parts; k += kThreads / 32) sum += p.partial[(int64_t)k * p.cols + c];
  s_sum[w][threadIdx.x % 32] = sum;
  __syncthreads();
  if (w != 0 || c >= p.cols) return;
#pragma unroll
  for (int k = 1; k < kThreads / 32; ++k) sum += s_sum[k][threadIdx.x];
  p.dgain[c] = p.accumulate ? p.dgain[c] + sum : sum;
}

namespace {

// The kernel of a row length: a warp per row up to 1024 columns, then CTAs.
static_assert(DOPT_NORM_MAX_COLS == 512 * 4 * 8, "the longest row's kernel");
template <typename T, template <typename, int, int> class Launch, typename P>
int launch_rows_t(P& p, cudaStream_t s, int* grid) {
  const int c = p.cols;
  if (c <= 256) return Launch<T, 32, 1>::run(p, s, grid);
  if (c <= 512) return Launch<T, 32, 2>::run(p, s, grid);
  if (c <= 1024) return Launch<T, 32, 4>::run(p, s, grid);
  if (c <= 2048) return Launch<T, 256, 1>::run(p, s, grid);
  if (c <= 4096) return Launch<T, 256, 2>::run(p, s, grid);
  if (c <= 8192) return Launch<T, 256, 4>::run(p, s, grid);
  return Launch<T, 512, 4>::run(p, s, grid);
}
template <template <typename, int, int> class Launch, typename P>
int launch_rows(int32_t dtype, P& p, cudaStream_t s, int* grid = nullptr) {
  return dtype == DOPT_F32    ? launch_rows_t<float, Launch>(p, s, grid)
         : dtype == DOPT_BF16 ? launch_rows_t<__nv_bfloat16, Launch>(p, s, grid)
                              : launch_rows_t<__half, Launch>(p, s, grid);
}

// As many CTAs as the device holds at once and the rows ask for.
template <auto Kern, int THREADS, int ROWS, typename P>
int row_grid(const P& p, int most, int* grid, const char* what) {
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
  *grid = (int)std::min<int64_t>({(int64_t)ctas, (int64_t)most, (p.rows + ROWS - 1) / ROWS});
  return DOPT_OK;
}

template <typename T, int G, int V>
struct Forward {
  static int run(const NormRows& p, cudaStream_t s, int*) {
    const char* what = "rms_norm launch";
    int grid = 0;
    if (int st = row_grid<rms_norm<T, G, V>, kRowThreads<G>, kRowsAtOnce<G>>(p, INT32_MAX, &grid, what)) return st;
    return launch_table<rms_norm<T, G, V>, 0, kRowThreads<G>>(p, s, what, false, grid);
  }
};
template <typename T, int G, int V>
struct Backward {
  static int run(const NormBackRows& p, cudaStream_t s, int* parts) {
    const char* what = "rms_norm_backward launch";
    int grid = 0;
    if (int st = row_grid<rms_norm_backward<T, G, V>, kRowThreads<G>, kRowsAtOnce<G>>(p, kMaxParts, &grid, what)) return st;
    *parts = grid;
    return launch_table<rms_norm_backward<T, G, V>, 0, kRowThreads<G>>(p, s, what, false, grid);
  }
};

int check_rows(const dopt_rows& r, int64_t cols, size_t elem, const char* name, const std::string& fn) {
  if (!aligned_to(r.data, elem)) return fail(DOPT_E_ALIGN, fn + name + " not aligned to its elements");
  if (r.data && r.ld < cols) return fail(DOPT_E_INVALID, fn + name + ": ld below cols");
  return DOPT_OK;
}

int check_norm(int64_t rows, int64_t cols, int32_t dtype, int32_t gain_dtype, const void* gain, const std::string& fn) {
  if (int st = check_sides(rows, cols, fn)) return st;
  if (cols > DOPT_NORM_MAX_COLS) return fail(DOPT_E_SIZE, fn + "more than " + std::to_string(DOPT_NORM_MAX_COLS) + " columns");
  if (!known_dtype(dtype)) return fail(DOPT_E_INVALID, fn + "unknown dtype");
  if (gain_dtype != DOPT_F32 && gain_dtype != dtype) return fail(DOPT_E_INVALID, fn + "the gain's dtype is fp32 or dtype");
  if (rows == 0 || cols == 0) return DOPT_OK;
  if (!gain) return fail(DOPT_E_INVALID, fn + "NULL gain");
  if (!aligned_to(gain, dtype_bytes(gain_dtype))) return fail(DOPT_E_ALIGN, fn + "gain not aligned to its elements");
  return DOPT_OK;
}

bool rows_vec(const dopt_rows& r, size_t elem) { return !r.data || eight_vectors(r.data, r.ld, elem); }

int parts_of(int64_t rows) { return (int)std::min<int64_t>(rows, kMaxParts); }

}  // namespace
}  // namespace dopt

using namespace dopt;

extern "C" {

int dopt_rms_norm(const dopt_rms_norm_args* a, dopt_stream stream) {
  return guard_entry([&]() -> int {
    const std::string fn = "dopt_rms_norm: ";
    if (!a) return fail(DOPT_E_INVALID, fn + "NULL arguments");
    int st = check_norm(a->rows, a->cols, a->dtype, a->gain_dtype, a->gain, fn);
    if (st) return st;
    if (!(a->eps >= 0.0) || std::isinf(a->eps)) return fail(DOPT_E_INVALID, fn + "bad eps");
    NormRows p{};
    uint32_t threshold;
    if ((st = check_drop(a->drop, &threshold, fn))) return st;
    if (a->y8 && (a->y8->rows != a->rows || a->y8->cols != a->cols))
      return fail(DOPT_E_INVALID, fn + "y8 has another size");
    if (a->rows == 0 || a->cols == 0) return DOPT_OK;
    if (!a->x.data) return fail(DOPT_E_INVALID, fn + "NULL x");
    if (!a->h.data && (a->residual.data || threshold)) return fail(DOPT_E_INVALID, fn + "NULL h with a residual or dropout");
    if (!a->y.data && !a->y8) return fail(DOPT_E_INVALID, fn + "neither y nor y8");
    const size_t elem = dtype_bytes(a->dtype);
    if ((st = check_rows(a->x, a->cols, elem, "x", fn))) return st;
    if ((st = check_rows(a->residual, a->cols, elem, "residual", fn))) return st;
    if ((st = check_rows(a->h, a->cols, elem, "h", fn))) return st;
    if ((st = check_rows(a->y, a->cols, elem, "y", fn))) return st;
    if (a->y8 && (st = check_matrix8(*a->y8, fn + "y8: "))) return st;
    if (!aligned_to(a->rstd, 4)) return fail(DOPT_E_ALIGN, fn + "rstd not aligned to its elements");
    p.x = RowsIn{a->x.data, a->x.ld};
    p.residual = RowsIn{a->residual.data, a->residual.ld};
    p.h = RowsOut{a->h.data, a->h.ld};
    p.y = RowsOut{a->y.data, a->y.ld};
    p.gain = a->gain;
    if (a->y8) {
      p.codes = a->y8->codes;
      p.scales = a->y8->scales;
      p.ld_codes = a->y8->ld;
    }
    p.rstd = a->rstd;
    p.rows = a->rows;
    p.cols = (int32_t)a->cols;
    p.groups = (uint32_t)scale_groups(a->cols);
    p.eps = (float)a->eps;
    p.drop = make_drop(a->drop, threshold);
    p.vec = rows_vec(a->x, elem) && rows_vec(a->residual, elem) && rows_vec(a->h, elem) && rows_vec(a->y, elem);
    p.gain_f32 = a->gain_dtype == DOPT_F32;
    return launch_rows<Forward>(a->dtype, p, (cudaStream_t)stream);
  });
}

size_t dopt_rms_norm_workspace_bytes(int64_t rows, int64_t cols) {
  const int st = guard_entry([&]() -> int {
    const std::string fn = "dopt_rms_norm_workspace_bytes: ";
    if (int bad = check_sides(rows, cols, fn)) return bad;
    return cols > DOPT_NORM_MAX_COLS ? fail(DOPT_E_SIZE, fn + "too many columns") : DOPT_OK;
  });
  return st ? 0 : std::max<size_t>(16, (size_t)parts_of(rows) * (size_t)cols * sizeof(float));
}

int dopt_rms_norm_backward(const dopt_rms_norm_backward_args* a, void* workspace, size_t workspace_bytes,
                           dopt_stream stream) {
  return guard_entry([&]() -> int {
    const std::string fn = "dopt_rms_norm_backward: ";
    if (!a) return fail(DOPT_E_INVALID, fn + "NULL arguments");
    int st = check_norm(a->rows, a->cols, a->dtype, a->gain_dtype, a->gain, fn);
    if (st) return st;
    NormBackRows p{};
    uint32_t threshold;
    if ((st = check_drop(a->drop, &threshold, fn))) return st;
    const cudaStream_t s = (cudaStream_t)stream;
    if (a->cols == 0) return DOPT_OK;
    if (!aligned_to(a->dgain, 4) || !aligned_to(a->rstd, 4))
      return fail(DOPT_E_ALIGN, fn + "dgain or rstd not aligned to its elements");
    if (a->rows == 0) {
      if (a->dgain && !a->accumulate) {
        const cudaError_t e = cudaMemsetAsync(a->dgain, 0, (size_t)a->cols * sizeof(float), s);
        if (e != cudaSuccess) return fail(DOPT_E_CUDA, fn + cudaGetErrorString(e));
      }
      return DOPT_OK;
    }
    if (!a->dy.data || !a->h.data || !a->rstd) return fail(DOPT_E_INVALID, fn + "NULL dy, h or rstd");
    if (!a->dh.data && !a->dx.data && !a->dgain) return fail(DOPT_E_INVALID, fn + "no output");
    if (a->dx.data && !threshold) return fail(DOPT_E_INVALID, fn + "dx without dropout (it is dh)");
    const size_t elem = dtype_bytes(a->dtype);
    if ((st = check_rows(a->dy, a->cols, elem, "dy", fn))) return st;
    if ((st = check_rows(a->h, a->cols, elem, "h", fn))) return st;
    if ((st = check_rows(a->dres, a->cols, elem, "dres", fn))) return st;
    if ((st = check_rows(a->dh, a->cols, elem, "dh", fn))) return st;
    if ((st = check_rows(a->dx, a->cols, elem, "dx", fn))) return st;
    if (a->dgain) {
      if (!workspace) return fail(DOPT_E_INVALID, fn + "NULL workspace");
      if (!aligned_to(workspace, 16)) return fail(DOPT_E_ALIGN, fn + "workspace not 16-byte aligned");
      const size_t need = dopt_rms_norm_workspace_bytes(a->rows, a->cols);
      if (workspace_bytes < need)
        return fail(DOPT_E_SIZE, fn + "workspace needs " + std::to_string(need) + " bytes, got " + std::to_string(workspace_bytes));
      p.partial = static_cast<float*>(workspace);
    }
    p.dy = RowsIn{a->dy.data, a->dy.ld};
    p.h = RowsIn{a->h.data, a->h.ld};
    p.dres = RowsIn{a->dres.data, a->dres.ld};
    p.dh = RowsOut{a->dh.data, a->dh.ld};
    p.dx = RowsOut{a->dx.data, a->dx.ld};
    p.gain = a->gain;
    p.rstd = a->rstd;
    p.rows = a->rows;
    p.cols = (int32_t)a->cols;
    p.drop = make_drop(a->drop, threshold);
    p.vec = rows_vec(a->dy, elem) && rows_vec(a->h, elem) && rows_vec(a->dres, elem) && rows_vec(a->dh, elem) && rows_vec(a->dx, elem);
    p.gain_f32 = a->gain_dtype == DOPT_F32;
    int parts = 0;
    if ((st = launch_rows<Backward>(a->dtype, p, s, &parts))) return st;
    if (!a->dgain) return DOPT_OK;
    GainParams g{p.partial, a->dgain, parts, p.cols, a->accumulate ? 1 : 0, 0};
    return launch_table<rms_norm_gain>(g, s, "rms_norm_gain launch", false, (p.cols + kGainColumns - 1) / kGainColumns);
  });
}

}  // extern "C"
