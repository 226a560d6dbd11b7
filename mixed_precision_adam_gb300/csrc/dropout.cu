// dropout.cu -- dropout with a mask from the counter-based generator of the
// 8-bit moments' rounding, and the residual's addition.
//
// The mask is recomputed wherever it is needed, from the element's number, so
// the backward pass is the same call on the gradient.
#include "matrix8.cuh"

namespace dopt {

struct DropoutParams {
  const void* x;
  const void* residual;
  void* y;
  int64_t n;
  Drop drop;
  int32_t n_tiles;
  bool vec;
};
constexpr int kDropTile = kThreads * 8;

template <typename T>
__global__ void __launch_bounds__(kThreads) dropout(const __grid_constant__ DropoutParams p) {
  const uint32_t key = drop_key(p.drop);
  for (int64_t t = blockIdx.x; t < p.n_tiles; t += gridDim.x) {
    const int64_t i = t * kDropTile + threadIdx.x * 8;
    const int n = (int)min((int64_t)8, p.n - i);
    if (n <= 0) continue;
    float f[8], r[8];
    load_some(static_cast<const T*>(p.x) + i, n, p.vec, f);
    if (p.residual) load_some(static_cast<const T*>(p.residual) + i, n, p.vec, r);
    if (p.drop.threshold) drop_eight(f, (uint64_t)i, p.drop, key);
    if (p.residual) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] += r[j];
    }
    store_some(static_cast<T*>(p.y) + i, n, p.vec, f);
  }
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
    p.x = a->x;
    p.residual = a->residual;
    p.y = a->y;
    p.n = a->numel;
    p.drop = make_drop(a->drop, threshold);
    p.n_tiles = (int32_t)tiles;
    p.vec = aligned_to(a->x, 16) && aligned_to(a->y, 16) && aligned_to(a->residual, 16);
    const cudaStream_t s = (cudaStream_t)stream;
    const char* what = "dropout launch";
    return a->dtype == DOPT_F32    ? launch_table<dropout<float>>(p, s, what)
           : a->dtype == DOPT_BF16 ? launch_table<dropout<__nv_bfloat16>>(p, s, what)
                                   : launch_table<dropout<__half>>(p, s, what);
  });
}
