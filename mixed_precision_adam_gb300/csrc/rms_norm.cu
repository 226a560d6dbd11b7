// rms_norm.cu -- the RMS norm with dropout and the residual's addition before
// it, values or 8-bit codes out, and the C entry points of the norm.
// 32768 x 4096 bf16 with a residual to codes: 150 us, 6.3 TB/s of 7 bytes per
// element (with dropout 190, bound by instructions); to values 169, 6.4 of 8,
// with dropout too.  16-bit rows off the vector grid take an access per
// element and run at half of that: 769 to 5501 columns 2.8 to 3.1 TB/s to
// codes, 3.6 to 4.3 to values.
#include <cfloat>
#include <initializer_list>

#include "rms_norm.cuh"

namespace dopt {

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
  double eps_wide;  // as it was given
  Drop drop;
  bool gain_f32;
};

template <bool WARP>
__device__ __noinline__ double row_sum_wide(double x, double (&s_sum)[kMaxRowThreads / 32]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  if constexpr (!WARP) {
    if (threadIdx.x % 32 == 0) s_sum[threadIdx.x / 32] = x;
    __syncthreads();
    x = s_sum[0];
    for (int w = 1; w < (int)blockDim.x / 32; ++w) x += s_sum[w];
    __syncthreads();
  }
  return x;
}

// The codes of a thread's eight values and their blocks' scale bytes.
template <bool VEC>
__device__ __forceinline__ void store_codes(const NormRows& p, int64_t row, int c, const float2 (&f)[4]) {
  uint8_t* dst = p.codes + row * p.ld_codes + c;
  if constexpr (VEC) {
    // a block of 128 columns is sixteen threads'
    uint32_t top = 0u;
#pragma unroll
    for (int k = 0; k < 4; ++k) top = top_of(top, f[k]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const BlockScale s(top);
    const uint2 code = make_uint2(four_codes(f[0], f[1], s), four_codes(f[2], f[3], s));
    if (c < p.cols) {
      *reinterpret_cast<uint2*>(dst) = code;
      if (threadIdx.x % 16 == 0) p.scales[scale_place(row, c / kBlock8, p.groups)] = (uint8_t)s.byte();
    }
  } else {
    // four values of every lane
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t top = top_of(top_of(0u, f[2 * q]), f[2 * q + 1]);
      const BlockScale s(__reduce_max_sync(0xFFFFFFFFu, top));
      const uint32_t code = four_codes(f[2 * q], f[2 * q + 1], s);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + 32 * (4 * q + j) < p.cols) dst[32 * (4 * q + j)] = (uint8_t)(code >> (8 * j));
      if (threadIdx.x % 32 == 0 && c + 128 * q < p.cols)
        p.scales[scale_place(row, (c + 128 * q) / kBlock8, p.groups)] = (uint8_t)s.byte();
    }
  }
}

// Whether a thread keeps the next row's values under this one's work: where
// their registers leave room.
template <typename T, int V>
constexpr bool kRowAhead = V * sizeof(T) <= 8;

// Threads and CTAs per SM that a kernel is compiled for (256 columns of bf16
// to 8 bits: 60 us with three CTAs, 72 with the two of 96 registers).
template <typename T, int V, bool VEC, int WARPS>
constexpr int kRowBound = WARPS == 0 ? 256 : kMaxRowThreads;
template <typename T, int V, bool VEC, int WARPS>
constexpr int kRowCtas = WARPS > 0 ? 1 : V == 1 ? 3 : 2;

template <typename T, int V, bool VEC, int WARPS>
__global__ void __launch_bounds__(kRowBound<T, V, VEC, WARPS>, kRowCtas<T, V, VEC, WARPS>) rms_norm(const __grid_constant__ NormRows p) {
  constexpr bool WARP = kWarpRows<WARPS>;
  __shared__ RowSums s_sum[2];
  __shared__ double s_wide[kMaxRowThreads / 32];
  using Piece = Eight8<T, VEC>;
  const RowShape<WARP> at;
  clear_sums<WARPS>(s_sum);
  const uint32_t key = drop_key(p.drop);
  const T* x = static_cast<const T*>(p.x.data);
  const T* residual = static_cast<const T*>(p.residual.data);
  const int64_t stride = at.stride();
  int64_t row = at.first();
  Piece xs[V], rs[V];
  auto load = [&](int64_t r) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = at.template column<V, VEC>(v);
      xs[v].load(x + r * p.x.ld + c, p.cols - c);
      if (residual) rs[v].load(residual + r * p.residual.ld + c, p.cols - c);
    }
  };
  if (row < p.rows) load(row);
  const RowGain<T, V, VEC, WARP, V <= 2 || (VEC && sizeof(T) == 2)> gain(p.gain, p.gain_f32, at, p.cols);
  int turn = 0;
  for (; row < p.rows; row += stride) {
    float2 f[V][4], squares = make_float2(0.f, 0.f);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = at.template column<V, VEC>(v);
      xs[v].widen8(f[v]);
      if (p.drop.threshold) drop_eight<VEC>(f[v], (uint64_t)row * p.cols + c, p.drop, key);
      if (residual) {
        float2 r[4];
        rs[v].widen8(r);
#pragma unroll
        for (int k = 0; k < 4; ++k) f[v][k] = __fadd2_rn(f[v][k], r[k]);
      }
      // what the norm sees is what is stored: the backward pass, and a norm
      // of h alone, then see the same
      round_eight<T>(f[v]);
    }
    if (kRowAhead<T, V> && row + stride < p.rows) load(row + stride);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = at.template column<V, VEC>(v);
      if (p.h.data) Piece::store(static_cast<T*>(p.h.data) + row * p.h.ld + c, p.cols - c, f[v]);
#pragma unroll
      for (int k = 0; k < 4; ++k) squares = __ffma2_rn(f[v][k], f[v][k], squares);
    }
    const float sum = row_sum<WARPS>(squares.x + squares.y, s_sum[turn]);
    turn ^= 1;
    const float m = sum / (float)p.cols + p.eps;
    float rstd, times, more = 1.f;  // h is multiplied by `times`, and by `more`
    if (m > 1e-30f && isfinite(m)) {
      rstd = rsqrtf(m);
      rstd *= fmaf(-0.5f * m * rstd, rstd, 1.5f);  // one step of Newton's method, as rsqrtf may be two last places off
      times = rstd;
    } else {
      // the squares left fp32's range, or what they lost below it may count:
      // up to 2^-149 each, 2^-49 of the bound above
      double wide = 0.0;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int k = 0; k < 4; ++k) wide += (double)f[v][k].x * (double)f[v][k].x + (double)f[v][k].y * (double)f[v][k].y;
      wide = row_sum_wide<WARP>(wide, s_wide);
      const double root = 1.0 / sqrt(wide / (double)p.cols + p.eps_wide);
      times = rstd = (float)root;
      if (root > (double)FLT_MAX && !isinf(root)) {
        // fp32 has no such number, but for h in two steps; the second is at
        // most 2^29 unless the row is zeros, which stay zeros
        times = 0x1p127f;
        more = (float)fmin(root * 0x1p-127, 0x1p30);
      }
    }
    if (at.g == 0 && p.rstd) p.rstd[row] = rstd;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = at.template column<V, VEC>(v);
      float2 w[4];
      gain.of(at, v, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) f[v][k] = __fmul2_rn(f[v][k], both_of(times));
      if (more != 1.f) {
#pragma unroll
        for (int k = 0; k < 4; ++k) f[v][k] = __fmul2_rn(f[v][k], both_of(more));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) f[v][k] = __fmul2_rn(f[v][k], w[k]);
      if (p.y.data) Piece::store(static_cast<T*>(p.y.data) + row * p.y.ld + c, p.cols - c, f[v]);
      if (p.codes) store_codes<VEC>(p, row, c, f[v]);
    }
    if (!kRowAhead<T, V> && row + stride < p.rows) load(row + stride);
  }
}

namespace {

template <typename T, int V, bool VEC, int WARPS>
int launch_one(const NormRows& p, cudaStream_t s) {
  const char* what = "rms_norm launch";
  constexpr int kRows = RowShape<kWarpRows<WARPS>>::kAtOnce;
  const int threads = row_threads<V, kWarpRows<WARPS>>(p.cols);
  int grid = 0;
  if (int st = row_grid<rms_norm<T, V, VEC, WARPS>>(threads, (p.rows + kRows - 1) / kRows, &grid, what)) return st;
  return launch_row_kernel<rms_norm<T, V, VEC, WARPS>>(p, grid, threads, s, what);
}
static_assert(DOPT_NORM_MAX_COLS <= kMaxRowThreads * 4 * 8, "the longest row's kernel");
// Eight columns per thread up to V = 4 times, in the fewest kernels that were
// best somewhere: few threads with much each for 16-bit vectors (4096 bf16
// columns to 8 bits: 59 us, with V = 2 67).
template <typename T, bool VEC>
int launch_length(const NormRows& p, cudaStream_t s) {
  const int c = p.cols;
  if (c <= 256) return launch_one<T, 1, VEC, 0>(p, s);
  if (c <= 512) return launch_one<T, 2, VEC, 0>(p, s);
  if constexpr (VEC && sizeof(T) == 2) {
    if (c <= 2048) return launch_one<T, 2, VEC, 8>(p, s);
    if (c <= 8192) return launch_one<T, 4, VEC, 8>(p, s);
  } else {
    if (c <= 4096) return launch_one<T, 2, VEC, 8>(p, s);
    if (c <= 8192) return launch_one<T, 2, VEC, 16>(p, s);
  }
  return launch_one<T, 4, VEC, 16>(p, s);
}
template <typename T>
int launch_norm(const NormRows& p, bool vec, cudaStream_t s) {
  return vec ? launch_length<T, true>(p, s) : launch_length<T, false>(p, s);
}

int check_rows(const dopt_rows& r, int64_t cols, size_t elem, const char* name, const std::string& fn) {
  if (!aligned_to(r.data, elem)) return fail(DOPT_E_ALIGN, fn + name + " not aligned to its elements");
  return r.data ? check_ld(r.ld, cols, fn + name + ": ") : DOPT_OK;
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

// The outputs of a call (those that are there) and what they share with each
// other and with the inputs.
struct NamedRows {
  const dopt_rows& r;
  const char* name;
};
int check_shared_rows(std::initializer_list<NamedRows> outputs, std::initializer_list<NamedRows> inputs, int64_t rows, int64_t cols,
                      size_t elem, const std::string& fn) {
  for (const NamedRows* a = outputs.begin(); a != outputs.end(); ++a) {
    const auto shared = [&](const NamedRows& b) { return shared_elements(a->r.data, a->r.ld, b.r.data, b.r.ld, rows, cols, elem); };
    for (const NamedRows* b = a + 1; b != outputs.end(); ++b)
      if (int st = check_shared(shared(*b), true, a->name, b->name, fn)) return st;
    for (const NamedRows& b : inputs)
      if (int st = check_shared(shared(b), false, a->name, b.name, fn)) return st;
  }
  return DOPT_OK;
}

bool rows_vec(const dopt_rows& r, size_t elem) { return !r.data || eight_vectors(r.data, r.ld, elem); }

int64_t parts_of(int64_t rows, int64_t cols) { return std::min<int64_t>(rows, max_parts(cols)); }

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
    if ((st = check_shared_rows({{a->h, "h"}, {a->y, "y"}}, {{a->x, "x"}, {a->residual, "residual"}}, a->rows, a->cols, elem, fn))) return st;
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
    p.eps_wide = a->eps;
    p.drop = make_drop(a->drop, threshold);
    const bool vec = a->cols % 8 == 0 && aligned_to(a->gain, 16) && rows_vec(a->x, elem) && rows_vec(a->residual, elem) && rows_vec(a->h, elem) && rows_vec(a->y, elem);
    p.gain_f32 = a->gain_dtype == DOPT_F32;
    const cudaStream_t s = (cudaStream_t)stream;
    return a->dtype == DOPT_F32    ? launch_norm<float>(p, vec, s)
           : a->dtype == DOPT_BF16 ? launch_norm<__nv_bfloat16>(p, vec, s)
                                   : launch_norm<__half>(p, vec, s);
  });
}

size_t dopt_rms_norm_workspace_bytes(int64_t rows, int64_t cols) {
  const int st = guard_entry([&]() -> int {
    const std::string fn = "dopt_rms_norm_workspace_bytes: ";
    if (int bad = check_sides(rows, cols, fn)) return bad;
    return cols > DOPT_NORM_MAX_COLS ? fail(DOPT_E_SIZE, fn + "too many columns") : DOPT_OK;
  });
  return st ? 0 : std::max<size_t>(16, (size_t)parts_of(rows, cols) * (size_t)cols * sizeof(float));
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
      if (a->dgain && !a->accumulate) return check_memset(cudaMemsetAsync(a->dgain, 0, (size_t)a->cols * sizeof(float), s), fn);
      return DOPT_OK;
    }
    if (!a->dy.data || !a->h.data || !a->rstd) return fail(DOPT_E_INVALID, fn + "NULL dy, h or rstd");
    if (!a->dh.data && !a->dx.data && !a->dgain) return fail(DOPT_E_INVALID, fn + "no output");
    const size_t elem = dtype_bytes(a->dtype);
    if ((st = check_rows(a->dy, a->cols, elem, "dy", fn))) return st;
    if ((st = check_rows(a->h, a->cols, elem, "h", fn))) return st;
    if ((st = check_rows(a->dres, a->cols, elem, "dres", fn))) return st;
    if ((st = check_rows(a->dh, a->cols, elem, "dh", fn))) return st;
    if ((st = check_rows(a->dx, a->cols, elem, "dx", fn))) return st;
    if ((st = check_shared_rows({{a->dh, "dh"}, {a->dx, "dx"}}, {{a->dy, "dy"}, {a->h, "h"}, {a->dres, "dres"}}, a->rows, a->cols, elem, fn)))
      return st;
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
    const bool vec = a->cols % 8 == 0 && aligned_to(a->gain, 16) && rows_vec(a->dy, elem) && rows_vec(a->h, elem) && rows_vec(a->dres, elem) && rows_vec(a->dh, elem) && rows_vec(a->dx, elem);
    p.gain_f32 = a->gain_dtype == DOPT_F32;
    int parts = 0;
    if ((st = launch_norm_backward(a->dtype, vec, p, s, &parts))) return st;
    return a->dgain ? launch_norm_gain(p.partial, parts, p.cols, a->dgain, a->accumulate != 0, s) : DOPT_OK;
  });
}

}  // extern "C"
