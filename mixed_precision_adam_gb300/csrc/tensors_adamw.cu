// tensors_adamw.cu -- AdamW over a list of tensors, moments in fp32.
#include "tensors.cuh"

namespace dopt {

template <typename PT, typename GT, int CAP>
__global__ void __launch_bounds__(kThreads) tensors_adamw(const __grid_constant__ AdamParamsT<CAP> p) {
  wait_for_prior_grids();
  if (p.found_inf && *p.found_inf) return;
  AdamScalars s;
  s.c = p.coef ? *p.coef : 1.f;
  s.step_size = p.dev ? p.dev->step_size : p.step_size;
  s.bc2_sqrt = p.dev ? p.dev->bc2_sqrt : p.bc2_sqrt;
  int si = -1;
  for (int t = blockIdx.x; t < p.n_tiles; t += gridDim.x) {
    const int k = si < 0 ? find_seg(p, t) : next_seg(p, si, t);
    const AdamSeg& sg = p.seg[k];
    if (k != si) s.decay = decay_of_seg(p, sg);
    si = k;
    const int64_t off = (int64_t)(t - sg.tile0) * kAdamTile;
    const int n = (int)min((int64_t)kAdamTile, sg.len - off);
    const GT* g = static_cast<const GT*>(sg.grad) + off;
    float* w = sg.weight + off;
    float* m = static_cast<float*>(sg.m) + off;
    float* v = static_cast<float*>(sg.v) + off;
    for (int e = threadIdx.x; e < n; e += kThreads) {
      float ww = w[e], mm = m[e], vv = v[e];
      adamw_element(widen<GT>(g[e]), p, s, ww, mm, vv);
      w[e] = ww;
      m[e] = mm;
      v[e] = vv;
      if constexpr (sizeof(PT) == 2) static_cast<PT*>(sg.param)[off + e] = narrow<PT>(ww);
    }
  }
}

template <typename PT, typename GT>
int launch_adamw_t(const AdamParamsT<kAdamCap>& p, cudaStream_t s) {
  if (p.n_seg <= kAdamSmallCap)
    return launch_table(tensors_adamw<PT, GT, kAdamSmallCap>, compact_table<AdamParamsT<kAdamSmallCap>, AdamHead>(p),
                        p.n_tiles, s, "tensors_adamw launch", nullptr, true);
  return launch_table(tensors_adamw<PT, GT, kAdamCap>, p, p.n_tiles, s, "tensors_adamw launch", nullptr, true);
}

int launch_tensors_adamw(int32_t param_dtype, int32_t grad_dtype, const AdamParamsT<kAdamCap>& p, cudaStream_t s) {
  const bool f32 = grad_dtype == DOPT_F32;
  switch (param_dtype) {
    case DOPT_BF16: return f32 ? launch_adamw_t<__nv_bfloat16, float>(p, s) : launch_adamw_t<__nv_bfloat16, __nv_bfloat16>(p, s);
    case DOPT_F16: return f32 ? launch_adamw_t<__half, float>(p, s) : launch_adamw_t<__half, __half>(p, s);
    default: return launch_adamw_t<float, float>(p, s);
  }
}

}  // namespace dopt
