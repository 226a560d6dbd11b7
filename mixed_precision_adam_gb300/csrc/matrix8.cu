// matrix8.cu -- matrices of values to 8-bit codes, their transposes likewise,
// and back.
//
// Bound by memory: fp32 values of a weight are read once and leave as 1 byte
// per orientation.  A CTA takes a 128 x 128 tile, so that both orientations'
// blocks end with the tile: a row's maximum is one warp's, a column's is
// gathered over the warps, and the transposed codes turn in shared memory, so
// that both are written in whole 128-byte lines.
#include "matrix8.cuh"

namespace dopt {

// One matrix in a launch.
struct MatrixSeg {
  void* values;
  uint8_t* codes;    // NULL: not asked for
  uint8_t* codes_t;
  uint8_t* scales;
  uint8_t* scales_t;
  int64_t ld, ld_out, ld_t;
  int32_t rows, cols;
  int32_t tile0;
  int32_t across;  // tiles per row of tiles
  int16_t square;
  int16_t vec;  // values are read four at a time
};
constexpr int kMatrixCap = 300, kMatrixSmallCap = 16;
struct MatrixHead {
  int32_t n_seg, n_tiles;
  DOPT_LIST_RECORD
};
template <int CAP>
struct MatrixParamsT : MatrixHead {
  MatrixSeg seg[CAP];
};
static_assert(sizeof(MatrixParamsT<kMatrixCap>) <= 32764, "kernel parameter limit");
enum : int { kSiteMatrix = 13 };

struct MatrixTile {
  int32_t r0, c0;      // first row and column
  int rows, cols;      // of the tile, 1 to 128
};
template <typename P>
__device__ __forceinline__ MatrixTile place_matrix_tile(const P& p, const MatrixSeg& sg, int t) {
  const uint32_t k = (uint32_t)(t - sg.tile0), down = k / (uint32_t)sg.across;
  MatrixTile a;
  a.r0 = (int32_t)(down * kBlock8);
  a.c0 = (int32_t)((k - down * sg.across) * kBlock8);
  a.rows = min(kBlock8, sg.rows - a.r0);
  a.cols = min(kBlock8, sg.cols - a.c0);
  if (!DOPT_TILE_OK(p, kSiteMatrix, a.r0, a.rows, sg.rows) || !DOPT_TILE_OK(p, kSiteMatrix, a.c0, a.cols, sg.cols))
    a.rows = 0;
  return a;
}

template <typename T>
__device__ __forceinline__ void load_four(const T* p, float* f);
template <>
__device__ __forceinline__ void load_four<float>(const float* p, float* f) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
}
template <>
__device__ __forceinline__ void load_four<__nv_bfloat16>(const __nv_bfloat16* p, float* f) {
  const uint2 a = __ldcs(reinterpret_cast<const uint2*>(p));
  f[0] = __uint_as_float(a.x << 16), f[1] = __uint_as_float(a.x & 0xFFFF0000u);
  f[2] = __uint_as_float(a.y << 16), f[3] = __uint_as_float(a.y & 0xFFFF0000u);
}
template <>
__device__ __forceinline__ void load_four<__half>(const __half* p, float* f) {
  const uint2 a = __ldcs(reinterpret_cast<const uint2*>(p));
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a.x));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&a.y));
  f[0] = x.x, f[1] = x.y, f[2] = y.x, f[3] = y.y;
}

// Warp w has rows 16 w to 16 w + 15 of a tile, lane l its columns 4 l to
// 4 l + 3: 64 values per thread, all of them loaded before the first is used.
constexpr int kRowsPerWarp = 16;
static_assert(kThreads / 32 * kRowsPerWarp == kBlock8, "a CTA has a tile's rows");

template <typename T, int CAP>
__global__ void __launch_bounds__(kThreads, 2) matrix8_pack(const __grid_constant__ MatrixParamsT<CAP> p) {
  __shared__ uint32_t s_top[kThreads / 32][kBlock8];  // largest of each column, by warp
  __shared__ uint32_t s_tile[kThreads / 32];          // and of all of the warp's values
  __shared__ uint4 s_turn[kBlock8 * kBlock8 / 16];    // transposed codes, 16 of a column at a time
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int hop = 1, si = 0;
  if ((int)blockIdx.x < p.n_tiles) si = find_seg(p, blockIdx.x);
  for (int t = blockIdx.x; t < p.n_tiles; t += gridDim.x) {
    si = next_seg(p, si, t, hop);
    const MatrixSeg& sg = p.seg[si];
    const MatrixTile a = place_matrix_tile(p, sg, t);
    const int n = a.cols - lane * 4;  // of this lane's columns
    float f[kRowsPerWarp][4];
    const T* src = static_cast<const T*>(sg.values) + (int64_t)(a.r0 + warp * kRowsPerWarp) * sg.ld + a.c0 + lane * 4;
#pragma unroll
    for (int k = 0; k < kRowsPerWarp; ++k) {
      const bool in = warp * kRowsPerWarp + k < a.rows;
      if (in && sg.vec && n >= 4) {
        load_four<T>(src + k * sg.ld, f[k]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) f[k][j] = in && j < n ? widen<T>(src[k * sg.ld + j]) : 0.f;
      }
    }
    uint32_t column[4] = {0u, 0u, 0u, 0u}, row[kRowsPerWarp], all = 0u;
#pragma unroll
    for (int k = 0; k < kRowsPerWarp; ++k) {
      uint32_t top = 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t b = __float_as_uint(f[k][j]) & 0x7FFFFFFFu;
        column[j] = max(column[j], b);
        top = max(top, b);
      }
      row[k] = top;
      all = max(all, top);
    }
    if (sg.square) {
      all = __reduce_max_sync(0xFFFFFFFFu, all);
      if (lane == 0) s_tile[warp] = all;
    } else if (sg.codes_t) {
      *reinterpret_cast<uint4*>(&s_top[warp][lane * 4]) = make_uint4(column[0], column[1], column[2], column[3]);
    }
    __syncthreads();
    uint32_t scale = 0u;
    if (sg.square) {
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) scale = max(scale, s_tile[w]);
      scale = m_scale_of(scale);
    }
    const float factor = code_factor(scale);
    if (sg.codes) {
      uint8_t* dst = sg.codes + (int64_t)(a.r0 + warp * kRowsPerWarp) * sg.ld_out + a.c0 + lane * 4;
      const uint32_t groups = (uint32_t)scale_groups(sg.cols);
#pragma unroll
      for (int k = 0; k < kRowsPerWarp; ++k) {
        const int r = warp * kRowsPerWarp + k;
        uint32_t s = scale;
        float up = factor;
        if (!sg.square) {
          s = m_scale_of(__reduce_max_sync(0xFFFFFFFFu, row[k]));
          up = code_factor(s);
        }
        if (r >= a.rows) continue;
        const uint32_t c = four_codes(f[k], up, s == 255u);
        if (n >= 4) {
          *reinterpret_cast<uint32_t*>(dst + k * sg.ld_out) = c;
        } else {
          for (int j = 0; j < n; ++j) dst[k * sg.ld_out + j] = (uint8_t)(c >> (8 * j));
        }
        if (lane == 0) sg.scales[scale_place(a.r0 + r, a.c0 / kBlock8, groups)] = (uint8_t)s;
      }
    }
    if (sg.codes_t) {
      const uint32_t groups = (uint32_t)scale_groups(sg.rows);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t s = scale;
        float up = factor;
        if (!sg.square) {
          uint32_t top = 0u;
#pragma unroll
          for (int w = 0; w < kThreads / 32; ++w) top = max(top, s_top[w][lane * 4 + j]);
          s = m_scale_of(top);
          up = code_factor(s);
        }
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float v[4] = {f[4 * q][j], f[4 * q + 1][j], f[4 * q + 2][j], f[4 * q + 3][j]};
          w[q] = four_codes(v, up, s == 255u);
        }
        // column 4 l + j holds eight pieces of 16 codes; turned by l so that
        // neither the lanes' writes here nor the reads below share banks
        s_turn[(lane * 4 + j) * 8 + ((warp + lane) & 7)] = make_uint4(w[0], w[1], w[2], w[3]);
        if (warp == 0 && j < n) sg.scales_t[scale_place(a.c0 + lane * 4 + j, a.r0 / kBlock8, groups)] = (uint8_t)s;
      }
      __syncthreads();
      // eight lanes write the 128 codes of a column
#pragma unroll
      for (int k = 0; k < kBlock8 * 8 / kThreads; ++k) {
        const int c = k * (kThreads / 8) + threadIdx.x / 8, piece = threadIdx.x % 8;
        if (c >= a.cols) continue;
        const uint4 v = s_turn[c * 8 + ((piece + (c >> 2)) & 7)];
        uint8_t* dst = sg.codes_t + (int64_t)(a.c0 + c) * sg.ld_t + a.r0 + piece * 16;
        const int m = a.rows - piece * 16;
        if (m >= 16) {
          *reinterpret_cast<uint4*>(dst) = v;
        } else {
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (j < m) dst[j] = (uint8_t)(w[j / 4] >> (8 * (j & 3)));
        }
      }
    }
    __syncthreads();  // the tile's shared arrays have been read
  }
}

// A warp has 16 rows of a tile, as above; lane l its columns 4 l to 4 l + 3.
template <typename T, int CAP>
__global__ void __launch_bounds__(kThreads, 2) matrix8_unpack(const __grid_constant__ MatrixParamsT<CAP> p) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int hop = 1, si = 0;
  if ((int)blockIdx.x < p.n_tiles) si = find_seg(p, blockIdx.x);
  for (int t = blockIdx.x; t < p.n_tiles; t += gridDim.x) {
    si = next_seg(p, si, t, hop);
    const MatrixSeg& sg = p.seg[si];
    const MatrixTile a = place_matrix_tile(p, sg, t);
    const int n = a.cols - lane * 4;
    const uint32_t groups = (uint32_t)scale_groups(sg.cols);
#pragma unroll 4
    for (int k = 0; k < kRowsPerWarp; ++k) {
      const int r = warp * kRowsPerWarp + k;
      if (r >= a.rows || n <= 0) continue;
      const int64_t at = (int64_t)(a.r0 + r) * sg.ld_out + a.c0 + lane * 4;
      const float unit = m_unit(sg.scales[scale_place(a.r0 + r, a.c0 / kBlock8, groups)]);
      uint2 c = make_uint2(0u, 0u);
      if (n >= 4) {
        c.x = *reinterpret_cast<const uint32_t*>(sg.codes + at);
      } else {
        for (int j = 0; j < n; ++j) c.x |= (uint32_t)sg.codes[at + j] << (8 * j);
      }
      float f[8];
      widen_codes(c, f);
      T* dst = static_cast<T*>(sg.values) + (int64_t)(a.r0 + r) * sg.ld + a.c0 + lane * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < n) dst[j] = narrow<T>(__fmul_rn(f[j], unit));
    }
  }
}

namespace {

template <auto Small, auto Big>
int launch_matrices(const MatrixParamsT<kMatrixCap>& p, cudaStream_t s, const char* what) {
  if (p.n_seg <= kMatrixSmallCap)
    return launch_table<Small>(compact_table<MatrixParamsT<kMatrixSmallCap>, MatrixHead>(p), s, what);
  return launch_table<Big>(p, s, what);
}
template <typename T>
int launch_pack(const MatrixParamsT<kMatrixCap>& p, cudaStream_t s) {
  return launch_matrices<matrix8_pack<T, kMatrixSmallCap>, matrix8_pack<T, kMatrixCap>>(p, s, "matrix8_pack launch");
}
template <typename T>
int launch_unpack(const MatrixParamsT<kMatrixCap>& p, cudaStream_t s) {
  return launch_matrices<matrix8_unpack<T, kMatrixSmallCap>, matrix8_unpack<T, kMatrixCap>>(p, s, "matrix8_unpack launch");
}

int64_t tiles_of(const dopt_matrix_values& m) { return row_blocks(m.rows) * row_blocks(m.cols); }

int check_matrices(const dopt_matrix_values* ms, int32_t n, bool pack, const char* fn) {
  if (n < 0) return fail(DOPT_E_INVALID, std::string(fn) + ": negative matrix count");
  if (n > 0 && !ms) return fail(DOPT_E_INVALID, std::string(fn) + ": NULL matrix list");
  int64_t tiles = 0;
  for (int32_t k = 0; k < n; ++k) {
    const dopt_matrix_values& m = ms[k];
    const std::string who = std::string(fn) + ": matrix " + std::to_string(k) + ": ";
    int st = check_sides(m.rows, m.cols, who);
    if (st) return st;
    if (!(pack ? known_dtype(m.values_dtype) : m.values_dtype == DOPT_F32 || m.values_dtype == DOPT_BF16))
      return fail(DOPT_E_INVALID, who + (pack ? "unknown values dtype" : "values are fp32 or bf16"));
    if (m.block != DOPT_BLOCK_ROW && m.block != DOPT_BLOCK_SQUARE) return fail(DOPT_E_INVALID, who + "unknown block");
    if (m.rows == 0 || m.cols == 0) continue;
    if ((tiles += tiles_of(m)) > INT32_MAX) return fail(DOPT_E_SIZE, who + "too many elements in the list");
    if (!m.values) return fail(DOPT_E_INVALID, who + "NULL values");
    if (!aligned_to(m.values, dtype_bytes(m.values_dtype)))
      return fail(DOPT_E_ALIGN, who + "values not aligned to their elements");
    if (m.ld < m.cols) return fail(DOPT_E_INVALID, who + "ld below cols");
    if (!m.out.codes && !(pack && m.out_t.codes)) return fail(DOPT_E_INVALID, who + "NULL codes");
    if (m.out.codes) {
      if (m.out.rows != m.rows || m.out.cols != m.cols) return fail(DOPT_E_INVALID, who + "out has another size");
      if ((st = check_matrix8(m.out, who + "out: "))) return st;
    }
    if (pack && m.out_t.codes) {
      if (m.out_t.rows != m.cols || m.out_t.cols != m.rows) return fail(DOPT_E_INVALID, who + "out_t has another size");
      if ((st = check_matrix8(m.out_t, who + "out_t: "))) return st;
    }
  }
  return DOPT_OK;
}

int run_matrices(const dopt_matrix_values* ms, int32_t n, bool pack, cudaStream_t s) {
  MatrixParamsT<kMatrixCap> p;
#if DOPT_BOUNDS_CHECK
  if (int st = bounds_record(&p.record)) return st;
#endif
  for (int32_t dt : {DOPT_F32, DOPT_BF16, DOPT_F16}) {
    p.n_seg = p.n_tiles = 0;
    auto flush = [&]() -> int {
      if (!p.n_seg) return DOPT_OK;
      const int st = !pack             ? (dt == DOPT_F32 ? launch_unpack<float>(p, s) : launch_unpack<__nv_bfloat16>(p, s))
                     : dt == DOPT_F32  ? launch_pack<float>(p, s)
                     : dt == DOPT_BF16 ? launch_pack<__nv_bfloat16>(p, s)
                                       : launch_pack<__half>(p, s);
      p.n_seg = p.n_tiles = 0;
      return st;
    };
    for (int32_t k = 0; k < n; ++k) {
      const dopt_matrix_values& m = ms[k];
      if (m.rows == 0 || m.cols == 0 || m.values_dtype != dt) continue;
      if (p.n_seg == kMatrixCap)
        if (int st = flush()) return st;
      const size_t elem = dtype_bytes(dt);
      MatrixSeg& g = p.seg[p.n_seg++];
      g = MatrixSeg{};
      g.values = m.values;
      g.codes = m.out.codes;
      g.scales = m.out.scales;
      if (pack) {
        g.codes_t = m.out_t.codes;
        g.scales_t = m.out_t.scales;
      }
      g.ld = m.ld;
      g.ld_out = m.out.ld;
      g.ld_t = m.out_t.ld;
      g.rows = (int32_t)m.rows;
      g.cols = (int32_t)m.cols;
      g.tile0 = p.n_tiles;
      g.across = (int32_t)row_blocks(m.cols);
      g.square = m.block == DOPT_BLOCK_SQUARE;
      g.vec = aligned_to(m.values, 4 * elem) && m.ld % 4 == 0;
      p.n_tiles += (int32_t)tiles_of(m);
    }
    if (int st = flush()) return st;
  }
  return DOPT_OK;
}

}  // namespace
}  // namespace dopt

using namespace dopt;

extern "C" {

int64_t dopt_matrix8_scale_bytes(int64_t rows, int64_t cols) {
  const int st = guard_entry([&] { return check_sides(rows, cols, "dopt_matrix8_scale_bytes: "); });
  return st ? st : scale_size(rows, cols);
}

int dopt_matrix8_pack(const dopt_matrix_values* matrices, int32_t n_matrices, dopt_stream stream) {
  return guard_entry([&]() -> int {
    const int st = check_matrices(matrices, n_matrices, true, "dopt_matrix8_pack");
    return st ? st : run_matrices(matrices, n_matrices, true, (cudaStream_t)stream);
  });
}

int dopt_matrix8_unpack(const dopt_matrix_values* matrices, int32_t n_matrices, dopt_stream stream) {
  return guard_entry([&]() -> int {
    const int st = check_matrices(matrices, n_matrices, false, "dopt_matrix8_unpack");
    return st ? st : run_matrices(matrices, n_matrices, false, (cudaStream_t)stream);
  });
}

}  // extern "C"
