// dropout.cu -- dropout with a mask from the counter-based generator of the
// 8-bit moments' rounding, and the residual's addition.
//
// The mask is recomputed wherever it is needed, from the element's number, so
// the backward pass is the same call on the gradient.  Bound by memory:
// 32768 x 4096 bf16 with a residual 117 us, 6.9 TB/s; without one 86, 6.2.
#include "matrix8.cuh"

namespace dopt {

struct DropoutParams {
  const void* x;
  const void* residual;
  void* y;
  int64_t n;
  Drop drop;
  int32_t n_tiles;
};
constexpr int kDropEights = 2;  // per thread
constexpr int kDropTile = kThreads * 8 * kDropEights;

// A CTA has a tile; a thread loads all of its elements before it uses one.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) dropout(const __grid_constant__ DropoutParams p) {
  const uint32_t key = drop_key(p.drop);
  const int64_t tile = (int64_t)blockIdx.x * kDropTile;
  const T* x = static_cast<const T*>(p.x);
  const T* residual = static_cast<const T*>(p.residual);
  T* y = static_cast<T*>(p.y);
  Eight8<T, VEC> a[kDropEights], r[kDropEights];
  int64_t at[kDropEights];
  int n[kDropEights];
#pragma unroll
  for (int v = 0; v < kDropEights; ++v) {
    at[v] = tile + v * kThreads * 8 + (VEC ? threadIdx.x * 8 : threadIdx.x / 32 * 256 + threadIdx.x % 32);
    n[v] = (int)max((int64_t)0, min((int64_t)256, p.n - at[v]));
    if (VEC && n[v] < 8) n[v] = 0;
    a[v].load(x + at[v], n[v]);
    if (residual) r[v].load(residual + at[v], n[v]);
  }
#pragma unroll
  for (int v = 0; v < kDropEights; ++v) {
    float2 f[4], g[4];
    a[v].widen8(f);
    if (p.drop.threshold) drop_eight<VEC>(f, (uint64_t)at[v], p.drop, key);
    if (residual) {
      r[v].widen8(g);
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = __fadd2_rn(f[k], g[k]);
    }
    Eight8<T, VEC>::store(y + at[v], n[v], f);
  }
  // fewer than eight elements at the end
  if (VEC && blockIdx.x == gridDim.x - 1 && threadIdx.x < (p.n & 7)) {
    const int64_t i = (p.n & ~(int64_t)7) + threadIdx.x;
    float f = widen<T>(x[i]);
    if (p.drop.threshold) {
      const uint32_t h = drop_hash((uint64_t)i >> 1, key);
      f = (i & 1 ? h >> 16 : h & 0xFFFFu) < p.drop.threshold ? 0.f : f * p.drop.keep;
    }
    if (residual) f += widen<T>(residual[i]);
    y[i] = narrow<T>(f);
  }
}

template <typename T>
int launch_dropout(const DropoutParams& p, bool vec, cudaStream_t s) {
  const char* what = "dropout launch";
  return vec ? launch_table<dropout<T, true>>(p, s, what, false, p.n_tiles) : launch_table<dropout<T, false>>(p, s, what, false, p.n_tiles);
}

}  // namespace dopt

using namespace dopt;

extern "C" int dopt_dropout(const dopt_dropout_args* a, dopt_stream stream) {
  return guard_entry([&]() -> int {
    const std::string fn = "dopt_dropout: ";
    if (!a) return fail(DOPT_E_INVALID, fn + "NULL arguments");
    if (a->numel < 0) return fail(DOPT_E_INVALID, fn + "negative numel");
    if (!known_dtype(a->dtype)) return fail(DOPT_E_INVALID, fn + "unknown dtype");
    DropoutParams p{};
    uint32_t threshold;
    if (int st = check_drop(a->drop, &threshold, fn)) return st;
    if (a->numel == 0) return DOPT_OK;
    const int64_t tiles = (a->numel - 1) / kDropTile + 1;
    if (tiles > INT32_MAX) return fail(DOPT_E_SIZE, fn + "too many elements");
    if (!a->x || !a->y) return fail(DOPT_E_INVALID, fn + "NULL x or y");
    const size_t elem = dtype_bytes(a->dtype);
    if (!aligned_to(a->x, elem) || !aligned_to(a->y, elem) || !aligned_to(a->residual, elem))
      return fail(DOPT_E_ALIGN, fn + "an array is not aligned to its elements");
    int st = check_shared(shared_elements(a->y, 0, a->x, 0, 1, a->numel, elem), false, "y", "x", fn);
    if (!st) st = check_shared(shared_elements(a->y, 0, a->residual, 0, 1, a->numel, elem), false, "y", "residual", fn);
    if (st) return st;
    p.x = a->x;
    p.residual = a->residual;
    p.y = a->y;
    p.n = a->numel;
    p.drop = make_drop(a->drop, threshold);
    p.n_tiles = (int32_t)tiles;
    const bool vec = aligned_to(a->x, 16) && aligned_to(a->y, 16) && aligned_to(a->residual, 16);
    const cudaStream_t s = (cudaStream_t)stream;
    return a->dtype == DOPT_F32    ? launch_dropout<float>(p, vec, s)
           : a->dtype == DOPT_BF16 ? launch_dropout<__nv_bfloat16>(p, vec, s)
                                   : launch_dropout<__half>(p, vec, s);
  });
}
