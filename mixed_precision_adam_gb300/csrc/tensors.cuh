// tensors.cuh -- what the kernels over a list of tensors share: the launch
// tables (a tensor's pointers, length and first tile, by value in the kernel
// parameters, as the run tables of the sharded step), typed loads and
// stores, the AdamW arithmetic, and the 8-bit moments' encoding.
//   tensors.cu        -- the C entry points: checks, tables, launches
//   tensors_norm.cu   -- the grad norm, and the finalize
//   tensors_adamw.cu  -- AdamW with fp32 moments
//   tensors_adamw8.cu -- AdamW with 8-bit moments, and their pack / unpack
// The 8-bit matrices (matrix8.cuh) take the encoding and the hash from here.
#pragma once

#include "kernels.cuh"

namespace dopt {

constexpr int kMomentBlock = DOPT_MOMENT_BLOCK;

// ------------------------------------------------------------ launch tables --

// One tensor's grad in a norm launch.
struct NormSeg {
  const void* grad;
  int64_t len;
  int32_t tile0;  // first tile of this tensor in the launch
  int16_t dtype;  // dopt_dtype of the grad
  int16_t shift;  // elements from the vector boundary below the first one to it
};
constexpr int kNormCap = 1280, kNormSmallCap = 64;
constexpr int kNormVector = 32;  // bytes: the grid tiles are cut on

// Debug builds (DOPT_BOUNDS_CHECK=1): every table carries the address of the
// record of tiles found outside their tensor (the first element at or past
// its end, or more elements than it has left); such a tile is skipped.
enum ListBoundsSite : int { kSiteListNorm = 9, kSiteListAdam = 10, kSiteListAdam8 = 11, kSiteListMoments = 12 };
#if DOPT_BOUNDS_CHECK
int bounds_record(unsigned long long** out);  // device address of the record on the current device
#define DOPT_LIST_RECORD unsigned long long* record;
#define DOPT_TILE_OK(p, site, lo, n, len) (::dopt::tile_ok((p).record, (site), (lo), (n), (len)))
__device__ __forceinline__ bool tile_ok(unsigned long long* record, int site, int64_t lo, int64_t n, int64_t len) {
  Extents x{};
  x.record = record;
  return range_ok(x, site, lo, n > 0 ? n : len + 1, len);  // a tile without elements has no place in a table
}
#else
#define DOPT_LIST_RECORD
#define DOPT_TILE_OK(p, site, lo, n, len) true
#endif

struct NormHead {
  Partial* partials;      // one slot per CTA of this launch
  int32_t* err_flag;      // the finalize's error word, which these kernels never set: cleared
  float inv_scale;
  int32_t n_seg, n_tiles;
  DOPT_LIST_RECORD
};
struct FinalizeParams {
  FinalizeArgs fin;
  int32_t n_tiles;  // 1: one CTA
};
template <int CAP>
struct NormParamsT : NormHead {
  NormSeg seg[CAP];
};
static_assert(sizeof(NormParamsT<kNormCap>) <= 32764, "kernel parameter limit");

// One tensor in an AdamW launch.
struct AdamSeg {
  void* param;
  const void* grad;
  float* weight;  // the fp32 weights: the master copy, or the fp32 param itself
  void* m;
  void* v;
  uint8_t* m_scale;
  uint8_t* v_scale;
  int64_t len;
  union {
    double wd_mult;  // device step scalars: the decay is formed on the device
    float decay;     // host step scalars: (float)(1 - lr * wd * wd_mult)
  };
  int32_t tile0;
  uint32_t key;  // 8-bit moments: the tensor's term of the rounding hash
  // Where the arrays have a common vector boundary: fp32 moments, elements
  // from the boundary below the tensor's first element to it (0 to 31);
  // 8-bit moments, 0 when the first element is one; -1: none.
  int32_t shift;
  int16_t param_dtype, grad_dtype;  // dopt_dtype
};
constexpr int kAdamCap = 360, kAdamSmallCap = 40;
constexpr int kAdamTile32 = 1024;  // elements per tile, fp32 moments
constexpr int kAdamTile = 2048;    // elements per tile, 8-bit moments

struct AdamHead {
  const float* coef;        // device scalar, or NULL: 1
  const int32_t* found_inf; // device flag, or NULL: never skipped
  const DevStep* dev;       // step scalars from the finalize pass, or NULL: the fields below
  const int64_t* d_step;    // with dev: the step number (already advanced to this step's)
  double lr_wd;
  float b1, b2, omb1, omb2, eps, step_size, bc2_sqrt;
  float inv_scale;
  uint32_t key;    // seed (+ the step's term, unless d_step)
  int32_t early;   // 1: this launch follows a kernel of the same call that writes none of its state
  int32_t n_seg, n_tiles;
  int32_t stride, span;  // see tile_walk
  DOPT_LIST_RECORD
};
template <int CAP>
struct AdamParamsT : AdamHead {
  AdamSeg seg[CAP];
};
static_assert(sizeof(AdamParamsT<kAdamCap>) <= 32764, "kernel parameter limit");
static_assert(sizeof(AdamParamsT<kAdamSmallCap>) <= 4096, "compact parameters");

// One tensor in a pack or unpack launch.
struct MomentSeg {
  void* m;  // values
  void* v;
  uint8_t* mc;  // codes
  uint8_t* vc;
  uint8_t* ms;  // scales
  uint8_t* vs;
  int64_t len;
  int32_t tile0;
  int32_t vec;  // 1: every array has the first element on a vector boundary
};
constexpr int kUnpackTile = 4096;  // elements per tile (pack: kAdamTile)
constexpr int kMomentCap = 500, kMomentSmallCap = 60;
struct MomentHead {
  int32_t n_seg, n_tiles;
  int32_t stride, span;  // see tile_walk
  DOPT_LIST_RECORD
};
template <int CAP>
struct MomentParamsT : MomentHead {
  MomentSeg seg[CAP];
};
static_assert(sizeof(MomentParamsT<kMomentCap>) <= 32764, "kernel parameter limit");

// The rounding hash's terms, as the header states them.
constexpr uint32_t kHashPair = 0x9E3779B9u, kHashTensor = 0x510E527Fu, kHashStep = 0x6A09E667u;
constexpr uint32_t kHashMul1 = 0xBB67AE85u, kHashMul2 = 0xA54FF53Bu;
__device__ __forceinline__ uint32_t hash_pair(uint32_t x) {
  uint64_t q = (uint64_t)x * kHashMul1;
  x = (uint32_t)q ^ (uint32_t)(q >> 32);
  q = (uint64_t)x * kHashMul2;
  return (uint32_t)q ^ (uint32_t)(q >> 32);
}

// A block's scale from the bits of its largest magnitude, 255 where that is
// not finite or above the largest code; and the number that e4m3 codes count
// under it.
__device__ __forceinline__ uint32_t exponent_of(uint32_t bits, uint32_t up) { return (bits + up) >> 23; }
__device__ __forceinline__ uint32_t m_scale_of(uint32_t top) {
  const uint32_t e = exponent_of(top, 0x1FFFFFu);
  return e >= 255u ? 255u : max((int)e - 8, 8);
}
__device__ __forceinline__ float m_unit(uint32_t s) {
  return s == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(s << 23);
}

// The tensor holding tile t among lo .. hi, by bisection.
template <typename P>
__device__ __forceinline__ int find_seg(const P& p, int t, int lo, int hi) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.seg[mid].tile0 <= t)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}
template <typename P>
__device__ __forceinline__ int find_seg(const P& p, int t) {
  return find_seg(p, t, 0, p.n_seg - 1);
}
// The same for a CTA's later tile, from the one before: in a large tensor the
// same one; among small tensors as many further on as the last time, nearly.
// `hop` keeps that number.  (Each entry read is a dependent load of the
// parameters: with plain bisections 1000 tensors of 50,000 elements took
// 193 us with 8-bit moments against 140, 253 with fp32 against 225.)
template <typename P>
__device__ __forceinline__ int next_seg(const P& p, int si, int t, int& hop) {
  if (si + 1 >= p.n_seg || p.seg[si + 1].tile0 > t) return si;
  const int guess = min(si + max(hop, 1), p.n_seg - 1);
  int found;
  if (p.seg[guess].tile0 <= t) {
    found = guess;
    if (guess + 1 < p.n_seg && p.seg[guess + 1].tile0 <= t) {
      found = guess + 1;
      if (guess + 2 < p.n_seg && p.seg[guess + 2].tile0 <= t) found = find_seg(p, t, guess + 2, p.n_seg - 1);
    }
  } else {
    found = p.seg[guess - 1].tile0 <= t ? guess - 1 : find_seg(p, t, si + 1, guess - 1);
  }
  hop = found - si;
  return found;
}

// The tiles of a CTA: from `first`, `stride` apart, below `end`.
struct TileWalk {
  int first, end;
};
template <typename P>
__device__ __forceinline__ TileWalk tile_walk(const P& p) {
  const int span = blockIdx.x / p.stride;
  TileWalk w;
  w.first = span * p.span + (int)blockIdx.x % p.stride;
  w.end = min(p.n_tiles, (span + 1) * p.span);
  return w;
}

// ------------------------------------------------------- elements by type --

template <typename T>
__device__ __forceinline__ float widen(T x);
template <>
__device__ __forceinline__ float widen<float>(float x) { return x; }
template <>
__device__ __forceinline__ float widen<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float widen<__half>(__half x) { return __half2float(x); }

template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half narrow<__half>(float x) { return __float2half_rn(x); }

// One element of an array whose type is known at run time.
__device__ __forceinline__ float load_element(const void* p, int64_t i, int dtype) {
  if (dtype == DOPT_F32) return static_cast<const float*>(p)[i];
  if (dtype == DOPT_BF16) return widen(static_cast<const __nv_bfloat16*>(p)[i]);
  return widen(static_cast<const __half*>(p)[i]);
}
// The 16-bit param of an fp32 weight (an fp32 param is the weight).
__device__ __forceinline__ void store_param(void* p, int64_t i, int dtype, float w) {
  if (dtype == DOPT_BF16) static_cast<__nv_bfloat16*>(p)[i] = narrow<__nv_bfloat16>(w);
  if (dtype == DOPT_F16) static_cast<__half*>(p)[i] = narrow<__half>(w);
}

// One element of AdamW, each operation rounded once in fp32: the arithmetic
// of the sharded step's AdamW pass.
struct AdamScalars {
  float c, decay, step_size, bc2_sqrt;
};
__device__ __forceinline__ void adamw_element(float g, const AdamHead& p, const AdamScalars& s, float& w, float& m,
                                              float& v) {
  g = __fmul_rn(__fmul_rn(g, p.inv_scale), s.c);
  w = __fmul_rn(w, s.decay);
  m = __fadd_rn(__fmul_rn(p.b1, m), __fmul_rn(p.omb1, g));
  v = __fadd_rn(__fmul_rn(p.b2, v), __fmul_rn(__fmul_rn(p.omb2, g), g));
  const float denom = __fadd_rn(__fdiv_rn(__fsqrt_rn(v), s.bc2_sqrt), p.eps);
  w = __fsub_rn(w, __fmul_rn(s.step_size, __fdiv_rn(m, denom)));
}

// The decoupled weight-decay factor of a tensor; in fp64, so out of line and
// once per tensor only when the step scalars live on the device.
static __device__ __noinline__ float tensor_decay(double lr_wd, double wd_mult) {
  return (float)(1.0 - lr_wd * wd_mult);
}
__device__ __forceinline__ float decay_of_seg(const AdamHead& p, const AdamSeg& sg) {
  return p.dev ? tensor_decay(p.dev->lr_wd, sg.wd_mult) : sg.decay;
}

// ----------------------------------------------------------- host launches --

// CTAs of a kernel that the current device holds at once, at most kMaxGrid.
// Asked once per device and kernel (its dynamic shared memory is allowed
// then too), so that a later launch, in a stream capture say, is only a launch.
template <auto Kern, size_t SMEM = 0>
int resident_ctas(int* out, const char* what) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(DOPT_E_CUDA, std::string("cudaGetDevice: ") + cudaGetErrorString(e));
  *out = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (*out) return DOPT_OK;
  if (SMEM) {
    e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM);
    if (e != cudaSuccess)
      return fail(DOPT_E_CUDA, std::string(what) + ": shared memory attribute: " + cudaGetErrorString(e));
  }
  int st = grid_for(Kern, kMaxGrid, out, SMEM);
  if (st) return st;
  if (dev < 64) known[dev].store(*out, std::memory_order_relaxed);
  return DOPT_OK;
}

// Launch of one kernel over a table.  A programmatic launch may start under
// the kernel before it (programmatic stream serialization): its CTAs wait
// for that grid before they read or write anything they may share with it.
// ctas: the grid; 0: as many as the tiles and the device ask for.
template <auto Kern, size_t SMEM = 0, int THREADS = kThreads, typename P>
int launch_table(const P& params, cudaStream_t s, const char* what, bool programmatic = false, int ctas = 0) {
  int grid = ctas;
  if (!ctas) {
    int st = resident_ctas<Kern, SMEM>(&grid, what);
    if (st) return st;
    grid = std::max(1, std::min(grid, params.n_tiles));
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = programmatic ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, Kern, params);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();  // reported here, not left for the next call to find
    return fail(DOPT_E_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
  }
  return check_launch(what);
}

// Sets a table's walk and launches it: the resident CTAs stride over the
// tiles, ROUNDS tiles each; then the next ones, started as they end, over the
// tiles after those.  CTAs that stride from the first tile to the last drift
// apart, and with them the pages that are being read and written: that cost
// 4 to 10 % on 1.35e9 elements, more the larger the list, with times that
// varied by as much.  A CTA's start costs more than its share of a few tiles,
// so each kernel has its own number of rounds.
template <auto Kern, size_t SMEM, int ROUNDS, typename P>
int launch_walk(P& params, cudaStream_t s, const char* what, bool programmatic) {
  int resident = 0;
  int st = resident_ctas<Kern, SMEM>(&resident, what);
  if (st) return st;
  params.stride = std::max(1, std::min(resident, params.n_tiles));
  params.span = params.stride * ROUNDS;
  const int spans = (params.n_tiles + params.span - 1) / params.span;
  return launch_table<Kern, SMEM>(params, s, what, programmatic, params.stride * std::max(1, spans));
}

// One launch each; the table's own count picks the compact parameter block.
int launch_tensors_norm(const NormParamsT<kNormCap>& p, cudaStream_t s);
int launch_tensors_finalize(const FinalizeArgs& fin, cudaStream_t s);
int tensors_norm_tile_bytes();
int tensors_norm_grid(const NormParamsT<kNormCap>& p, int* grid);  // that launch's CTAs
int launch_tensors_adamw(AdamParamsT<kAdamCap>& p, cudaStream_t s);
int launch_tensors_adamw8(AdamParamsT<kAdamCap>& p, cudaStream_t s);
int launch_state8_pack(int32_t values_dtype, MomentParamsT<kMomentCap>& p, cudaStream_t s);
int launch_state8_unpack(int32_t values_dtype, MomentParamsT<kMomentCap>& p, cudaStream_t s);

// A table's parameters with room for CAP entries only.
template <typename Small, typename Head, typename Big>
Small compact_table(const Big& b) {
  Small out{};
  static_cast<Head&>(out) = static_cast<const Head&>(b);
  for (int i = 0; i < b.n_seg; ++i) out.seg[i] = b.seg[i];
  return out;
}

}  // namespace dopt
