// matrix8.cu -- matrices of values to 8-bit codes, their transposes likewise,
// and back.
//
// Bound by memory: fp32 values of a weight are read once and leave as 1 byte
// per orientation.  A CTA takes a 128 x 128 tile, so that both orientations'
// blocks end with the tile: a row's maximum is one warp's, a column's is
// gathered over the warps, and the transposed codes turn in shared memory, so
// that both are written in whole 128-byte lines.  Measured: 32768 x 4096 bf16
// in rows both ways 98 us, 5.5 TB/s of 4 bytes per element (its instructions:
// 77 % of the issue slots), 11008 x 4096 fp32 in squares both ways 53 us, 5.1
// TB/s; back to bf16 66 us for 32768 x 4096, 6.1 TB/s.
#include <type_traits>

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
  int16_t vec;  // the values' rows allow vectors
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

// Four consecutive values of a row as they are loaded, their magnitudes' bits
// (in the type's own format, which orders them) and what those are in fp32.
template <typename T>
struct Four {  // 16-bit types
  uint2 r;
  __device__ __forceinline__ void load(const T* p) { r = __ldcs(reinterpret_cast<const uint2*>(p)); }
  // from shared memory
  __device__ __forceinline__ void take(const T* p) { r = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void zero() { r = make_uint2(0u, 0u); }
  __device__ __forceinline__ float2 low() const { return widen_pair<T>(r.x); }
  __device__ __forceinline__ float2 high() const { return widen_pair<T>(r.y); }
  // Element j alone.
  __device__ __forceinline__ float at(int j) const {
    const float2 x = widen_pair<T>(j < 2 ? r.x : r.y);
    return j & 1 ? x.y : x.x;
  }
  struct Top {  // of each of the four; NaN where one is
    uint32_t lo = 0u, hi = 0u;
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
      using Pair = std::conditional_t<std::is_same<T, __half>::value, __half2, __nv_bfloat162>;
      const Pair m = __hmax2_nan(*reinterpret_cast<const Pair*>(&a), __habs2(*reinterpret_cast<const Pair*>(&b)));
      return *reinterpret_cast<const uint32_t*>(&m);
    }
    __device__ __forceinline__ void add(const Four& v) {
      lo = larger(lo, v.r.x);
      hi = larger(hi, v.r.y);
    }
    __device__ __forceinline__ uint32_t all() const {
      const uint32_t m = larger(lo, hi);
      return max(m & 0xFFFFu, m >> 16);
    }
    __device__ __forceinline__ uint4 each() const { return make_uint4(lo & 0xFFFFu, lo >> 16, hi & 0xFFFFu, hi >> 16); }
  };
  static __device__ __forceinline__ uint32_t fp32_bits(uint32_t top) { return __float_as_uint(widen_pair<T>(top).x); }
};
template <>
struct Four<float> {
  float4 r;
  __device__ __forceinline__ void load(const float* p) { r = __ldcs(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ void take(const float* p) { r = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void zero() { r = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ float2 low() const { return make_float2(r.x, r.y); }
  __device__ __forceinline__ float2 high() const { return make_float2(r.z, r.w); }
  __device__ __forceinline__ float at(int j) const { return j == 0 ? r.x : j == 1 ? r.y : j == 2 ? r.z : r.w; }
  struct Top {
    uint4 t = make_uint4(0u, 0u, 0u, 0u);
    __device__ __forceinline__ void add(const Four& v) {
      t.x = max(t.x, __float_as_uint(v.r.x) & 0x7FFFFFFFu);
      t.y = max(t.y, __float_as_uint(v.r.y) & 0x7FFFFFFFu);
      t.z = max(t.z, __float_as_uint(v.r.z) & 0x7FFFFFFFu);
      t.w = max(t.w, __float_as_uint(v.r.w) & 0x7FFFFFFFu);
    }
    __device__ __forceinline__ uint32_t all() const { return max(max(t.x, t.y), max(t.z, t.w)); }
    __device__ __forceinline__ uint4 each() const { return t; }
  };
  static __device__ __forceinline__ uint32_t fp32_bits(uint32_t top) { return top; }
};

// A warp has consecutive rows of a tile, 16 of 16-bit values and 8 of fp32
// ones, lane l its columns 4 l to 4 l + 3: 128 bytes per thread, all of them
// loaded before the first is used.
template <typename T>
struct PackShape {
  static constexpr int kRows = sizeof(T) == 2 ? 16 : 8;
  static constexpr int kWarps = kBlock8 / kRows, kThreads = kWarps * 32;
  static constexpr int kCtas = sizeof(T) == 2 ? 4 : 2;  // per SM: what the values' registers allow
};

// The codes of a warp's rows (`rows` of them, `n` of this lane's columns),
// 128 bytes of a row at a time, and their scale bytes.
template <typename T, bool WHOLE>
__device__ __forceinline__ void store_rows(const MatrixSeg& sg, const Four<T> (&f)[PackShape<T>::kRows], const BlockScale& square,
                                           int64_t r0, int32_t c0, int rows, int n) {
  constexpr int kRows = PackShape<T>::kRows;
  const int lane = threadIdx.x % 32;
  uint8_t* dst = sg.codes + r0 * sg.ld_out + c0 + lane * 4;
  uint32_t mine = 0u;  // lane k: the bits of row k's largest
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    BlockScale sc = square;
    if (!sg.square) {
      typename Four<T>::Top row;
      row.add(f[k]);
      const uint32_t top = Four<T>::fp32_bits(__reduce_max_sync(0xFFFFFFFFu, row.all()));
      sc = BlockScale(top);
      if (lane == k) mine = top;
    }
    uint32_t c = four_codes(f[k].low(), f[k].high(), sc.up());
    if (sc.nan) c = 0u;
    if (WHOLE || (k < rows && n >= 4)) {
      __stcs(reinterpret_cast<uint32_t*>(dst), c);
    } else if (k < rows) {
      for (int j = 0; j < n; ++j) dst[j] = (uint8_t)(c >> (8 * j));
    }
    dst += sg.ld_out;
  }
  if (lane < (WHOLE ? kRows : rows))
    sg.scales[scale_place(r0 + lane, c0 / kBlock8, (uint32_t)scale_groups(sg.cols))] =
        (uint8_t)(sg.square ? square : BlockScale(mine)).byte();
}

// A CTA per tile: the next ones' loads then run under this one's stores.
template <typename T, int CAP>
__global__ void __launch_bounds__(PackShape<T>::kThreads, PackShape<T>::kCtas) matrix8_pack(const __grid_constant__ MatrixParamsT<CAP> p) {
  constexpr int kRows = PackShape<T>::kRows, kWarps = PackShape<T>::kWarps, kPackThreads = PackShape<T>::kThreads;
  __shared__ alignas(16) uint32_t s_top[kWarps][kBlock8];  // largest of each column, by warp; then, first, of all
  __shared__ uint32_t s_tile[kWarps];                      // and of all of the warp's values
  // values on their way to their lanes, a few rows of a warp at a time; then
  // the transposed codes, a warp's of a column at a time
  constexpr int kStageRows = sizeof(T) == 2 ? 8 : 4;
  __shared__ union alignas(16) {
    T stage[kWarps][kStageRows][kBlock8];
    uint32_t turn[kBlock8 * kBlock8 / 4];
  } s;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const MatrixSeg& sg = p.seg[find_seg(p, blockIdx.x)];
  const MatrixTile a = place_matrix_tile(p, sg, blockIdx.x);
  const int rows = min(kRows, a.rows - warp * kRows);  // of the warp
  const int64_t r0 = (int64_t)a.r0 + warp * kRows;
  const bool whole = a.rows == kBlock8 && a.cols == kBlock8;
  Four<T> f[kRows];
  const T* src = static_cast<const T*>(sg.values) + r0 * sg.ld + a.c0;
  if (sg.vec && whole) {
    src += lane * 4;
#pragma unroll
    for (int k = 0; k < kRows; ++k, src += sg.ld) f[k].load(src);
  } else {
    // consecutive lanes load consecutive elements, and take four through
    // shared memory
#pragma unroll
    for (int part = 0; part < kRows; part += kStageRows) {
      T t[kStageRows][4];
#pragma unroll
      for (int k = 0; k < kStageRows; ++k, src += sg.ld)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = lane + 32 * j;
          t[k][j] = part + k < rows && c < a.cols ? __ldcs(src + c) : narrow<T>(0.f);
        }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < kStageRows; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) s.stage[warp][k][lane + 32 * j] = t[k][j];
      __syncwarp();
#pragma unroll
      for (int k = 0; k < kStageRows; ++k) f[part + k].take(&s.stage[warp][k][lane * 4]);
    }
  }
  uint32_t top = 0u;  // square: of the tile
  if (sg.square || sg.codes_t) {
    typename Four<T>::Top column;
#pragma unroll
    for (int k = 0; k < kRows; ++k) column.add(f[k]);
    if (sg.square) {
      const uint32_t all = __reduce_max_sync(0xFFFFFFFFu, column.all());
      if (lane == 0) s_tile[warp] = all;
    } else {
      *reinterpret_cast<uint4*>(&s_top[warp][lane * 4]) = column.each();
    }
    __syncthreads();
    if (sg.square) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = max(top, s_tile[w]);
    } else if (threadIdx.x < kBlock8) {
      // a thread per column, which the lanes that have it read together below
      uint32_t t = 0u;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) t = max(t, s_top[w][threadIdx.x]);
      s_top[0][threadIdx.x] = t;
    }
  }
  const BlockScale square(Four<T>::fp32_bits(top));
  if (sg.codes) {
    if (whole)
      store_rows<T, true>(sg, f, square, r0, a.c0, kRows, 4);
    else
      store_rows<T, false>(sg, f, square, r0, a.c0, rows, a.cols - lane * 4);
  }
  if (!sg.codes_t) return;
  uint4 tops = make_uint4(top, top, top, top);
  if (!sg.square) {
    __syncthreads();
    tops = *reinterpret_cast<const uint4*>(&s_top[0][lane * 4]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const BlockScale sc(Four<T>::fp32_bits(j == 0 ? tops.x : j == 1 ? tops.y : j == 2 ? tops.z : tops.w));
    uint32_t w[kRows / 4];
#pragma unroll
    for (int q = 0; q < kRows / 4; ++q) {
      w[q] = four_codes(make_float2(f[4 * q].at(j), f[4 * q + 1].at(j)), make_float2(f[4 * q + 2].at(j), f[4 * q + 3].at(j)), sc.up());
      if (sc.nan) w[q] = 0u;
    }
    // a column's 128 codes are turned by 16 l, so that the lanes' writes here
    // spread over the banks and 16 codes stay together
    uint32_t* at = &s.turn[(lane * 4 + j) * 32 + ((warp * (kRows / 4) + 4 * lane) & 31)];
    if constexpr (kRows == 16)
      *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
    else
      *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
    if (warp == j && lane * 4 + j < a.cols && a.rows > 0)
      sg.scales_t[scale_place((int64_t)a.c0 + lane * 4 + j, a.r0 / kBlock8, (uint32_t)scale_groups(sg.rows))] =
          (uint8_t)sc.byte();
  }
  __syncthreads();
  // eight lanes write the 128 codes of a column
#pragma unroll
  for (int k = 0; k < kBlock8 * 8 / kPackThreads; ++k) {
    const int c = k * (kPackThreads / 8) + threadIdx.x / 8, piece = threadIdx.x % 8;
    if (c >= a.cols) continue;
    const uint4 v = *reinterpret_cast<const uint4*>(&s.turn[c * 32 + ((4 * piece + 4 * (c >> 2)) & 31)]);
    uint8_t* dst = sg.codes_t + ((int64_t)a.c0 + c) * sg.ld_t + a.r0 + piece * 16;
    const int m = a.rows - piece * 16;
    if (m >= 16) {
      __stcs(reinterpret_cast<uint4*>(dst), v);
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (j < m) dst[j] = (uint8_t)(w[j / 4] >> (8 * (j & 3)));
    }
  }
}

// Warp w has 16 rows of a tile.  Where the values can be written
// in vectors a lane has 16 codes of every fourth row; else four of each row,
// which go to the lanes that make consecutive elements of them.
constexpr int kUnpackRows = kBlock8 / (kThreads / 32);
template <typename T, int CAP>
__global__ void __launch_bounds__(kThreads, 4) matrix8_unpack(const __grid_constant__ MatrixParamsT<CAP> p) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const MatrixSeg& sg = p.seg[find_seg(p, blockIdx.x)];
  const MatrixTile a = place_matrix_tile(p, sg, blockIdx.x);
  const int rows = min(kUnpackRows, a.rows - warp * kUnpackRows);
  if (rows <= 0) return;
  const int64_t r0 = (int64_t)a.r0 + warp * kUnpackRows;
  const uint32_t groups = (uint32_t)scale_groups(sg.cols), block = a.c0 / kBlock8;
  const uint8_t* codes = sg.codes + r0 * sg.ld_out + a.c0;
  T* values = static_cast<T*>(sg.values) + r0 * sg.ld + a.c0;
  // lane k: row k's scale
  const uint32_t scale = lane < rows ? sg.scales[scale_place(r0 + lane, block, groups)] : 0u;
  if (sg.vec && a.cols == kBlock8) {
    const int c = lane % 8 * 16;
    uint4 code[kUnpackRows / 4];
#pragma unroll
    for (int k = 0; k < kUnpackRows / 4; ++k) {
      const int r = lane / 8 + 4 * k;
      if (r < rows) code[k] = __ldcs(reinterpret_cast<const uint4*>(codes + r * sg.ld_out + c));
    }
#pragma unroll
    for (int k = 0; k < kUnpackRows / 4; ++k) {
      const int r = lane / 8 + 4 * k;
      const float unit = m_unit(__shfl_sync(0xFFFFFFFFu, scale, r));
      if (r >= rows) continue;
      T* dst = values + r * sg.ld + c;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float2 f[4];
        widen_codes(q ? make_uint2(code[k].z, code[k].w) : make_uint2(code[k].x, code[k].y), f);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = __fmul2_rn(f[j], both_of(unit));
        Eight8<T, true>::store(dst + 8 * q, 8, f);
      }
    }
    return;
  }
  const int n = a.cols - lane * 4;
  uint32_t code[kUnpackRows];
#pragma unroll
  for (int k = 0; k < kUnpackRows; ++k) {
    code[k] = 0u;
    if (k >= rows) continue;
    const uint8_t* src = codes + k * sg.ld_out + lane * 4;
    if (n >= 4)
      code[k] = __ldcs(reinterpret_cast<const uint32_t*>(src));
    else
      for (int j = 0; j < n; ++j) code[k] |= (uint32_t)src[j] << (8 * j);
  }
#pragma unroll
  for (int k = 0; k < kUnpackRows; ++k) {
    if (k >= rows) break;
    const float unit = m_unit(__shfl_sync(0xFFFFFFFFu, scale, k));
    // the codes of columns l, l + 32, l + 64 and l + 96, from lanes l / 4, ...
    uint32_t mine = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      mine |= (__shfl_sync(0xFFFFFFFFu, code[k], lane / 4 + 8 * j) >> (8 * (lane & 3)) & 0xFFu) << (8 * j);
    float2 f[4];
    widen_codes(make_uint2(mine, 0u), f);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (lane + 32 * j < a.cols)
        __stcs(values + k * sg.ld + lane + 32 * j, narrow<T>(__fmul_rn(j & 1 ? f[j / 2].y : f[j / 2].x, unit)));
  }
}

namespace {

template <auto Small, auto Big, int THREADS>
int launch_matrices(const MatrixParamsT<kMatrixCap>& p, cudaStream_t s, const char* what) {
  if (p.n_seg <= kMatrixSmallCap)
    return launch_table<Small, 0, THREADS>(compact_table<MatrixParamsT<kMatrixSmallCap>, MatrixHead>(p), s, what, false,
                                                  p.n_tiles);
  return launch_table<Big, 0, THREADS>(p, s, what, false, p.n_tiles);
}
template <typename T>
int launch_pack(const MatrixParamsT<kMatrixCap>& p, cudaStream_t s) {
  return launch_matrices<matrix8_pack<T, kMatrixSmallCap>, matrix8_pack<T, kMatrixCap>, PackShape<T>::kThreads>(p, s, "matrix8_pack launch");
}
template <typename T>
int launch_unpack(const MatrixParamsT<kMatrixCap>& p, cudaStream_t s) {
  return launch_matrices<matrix8_unpack<T, kMatrixSmallCap>, matrix8_unpack<T, kMatrixCap>, kThreads>(p, s, "matrix8_unpack launch");
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
    if ((st = check_ld(m.ld, m.cols, who))) return st;
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
      // packing reads four values at a time, unpacking writes 16 bytes
      g.vec = pack ? aligned_to(m.values, 4 * elem) && m.ld % 4 == 0 : eight_vectors(m.values, m.ld, elem);
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
