// tensors.cu -- the C entry points of the optimizer step over a list of
// tensors: argument checks, the launch tables and the launches.
#include <cmath>
#include <new>

#include "tensors.cuh"

namespace {
using namespace dopt;

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t dtype_bytes(int32_t dtype) { return dtype == DOPT_F32 ? 4 : 2; }
bool known_dtype(int32_t dtype) { return dtype == DOPT_F32 || dtype == DOPT_BF16 || dtype == DOPT_F16; }

std::string at(const char* fn, int32_t k) { return std::string(fn) + ": tensor " + std::to_string(k) + ": "; }

int64_t tiles_of(int64_t numel, int tile) { return numel / tile + (numel % tile != 0); }

// Adds a tensor's tiles (of the smallest size used, with one to spare) to a
// list's count; false when a launch could not number them (2e12 elements).
bool count_tiles(int64_t numel, int64_t* total) {
  *total += tiles_of(numel, 1024) + 1;
  return *total <= INT32_MAX;
}

int check_list(const void* tensors, int32_t n, const char* fn) {
  if (n < 0) return fail(DOPT_E_INVALID, std::string(fn) + ": negative tensor count");
  if (n > 0 && !tensors) return fail(DOPT_E_INVALID, std::string(fn) + ": NULL tensor list");
  return DOPT_OK;
}

// One array of tensor k: present, and aligned to its elements.
int check_array(const void* p, size_t elem, const char* name, int32_t k, const char* fn) {
  if (!p) return fail(DOPT_E_INVALID, at(fn, k) + "NULL " + name);
  if (!aligned_to(p, elem)) return fail(DOPT_E_ALIGN, at(fn, k) + name + " not aligned to its elements");
  return DOPT_OK;
}

int check_grads(const dopt_tensor* ts, int32_t n, const char* fn) {
  int st = check_list(ts, n, fn);
  if (st) return st;
  int64_t tiles = 0;
  for (int32_t k = 0; k < n; ++k) {
    const dopt_tensor& t = ts[k];
    if (t.numel < 0) return fail(DOPT_E_INVALID, at(fn, k) + "negative numel");
    if (!known_dtype(t.grad_dtype)) return fail(DOPT_E_INVALID, at(fn, k) + "unknown grad dtype");
    if (t.numel == 0) continue;
    if (!count_tiles(t.numel, &tiles)) return fail(DOPT_E_SIZE, at(fn, k) + "too many elements in the list");
    if ((st = check_array(t.grad, dtype_bytes(t.grad_dtype), "grad", k, fn))) return st;
  }
  return DOPT_OK;
}

int check_states(const dopt_tensor* ts, int32_t n, const char* fn) {
  int st = check_grads(ts, n, fn);
  if (st) return st;
  for (int32_t k = 0; k < n; ++k) {
    const dopt_tensor& t = ts[k];
    if (!known_dtype(t.param_dtype)) return fail(DOPT_E_INVALID, at(fn, k) + "unknown param dtype");
    if (t.grad_dtype != DOPT_F32 && t.grad_dtype != t.param_dtype)
      return fail(DOPT_E_INVALID, at(fn, k) + "the grad dtype must be the param dtype or fp32");
    if (t.moments != DOPT_MOMENTS_F32 && t.moments != DOPT_MOMENTS_8BIT)
      return fail(DOPT_E_INVALID, at(fn, k) + "unknown moments format");
    if (!std::isfinite(t.wd_mult)) return fail(DOPT_E_INVALID, at(fn, k) + "wd_mult is not finite");
    if (t.numel == 0) continue;
    const size_t moment = t.moments == DOPT_MOMENTS_F32 ? 4 : 1;
    if ((st = check_array(t.param, dtype_bytes(t.param_dtype), "param", k, fn))) return st;
    if (t.param_dtype == DOPT_F32 && t.master)
      return fail(DOPT_E_INVALID, at(fn, k) + "master must be NULL for an fp32 param (the param is the master)");
    if (t.param_dtype != DOPT_F32 && (st = check_array(t.master, 4, "master", k, fn))) return st;
    if ((st = check_array(t.exp_avg, moment, "exp_avg", k, fn))) return st;
    if ((st = check_array(t.exp_avg_sq, moment, "exp_avg_sq", k, fn))) return st;
    if (t.moments == DOPT_MOMENTS_8BIT && (!t.exp_avg_scale || !t.exp_avg_sq_scale))
      return fail(DOPT_E_INVALID, at(fn, k) + "8-bit moments need their scales");
    if (t.moments == DOPT_MOMENTS_F32 && (t.exp_avg_scale || t.exp_avg_sq_scale))
      return fail(DOPT_E_INVALID, at(fn, k) + "fp32 moments have no scales");
  }
  return DOPT_OK;
}

int check_hp(const dopt_adamw_hparams* hp, bool device_step, float inv_scale, const char* fn) {
  if (!hp) return fail(DOPT_E_INVALID, std::string(fn) + ": NULL hparams");
  const bool ok = (device_step || hp->step >= 1) && std::isfinite(hp->lr) && hp->lr >= 0 && hp->beta1 >= 0 && hp->beta1 < 1 &&
                  hp->beta2 >= 0 && hp->beta2 < 1 && std::isfinite(hp->eps) && hp->eps > 0 &&
                  std::isfinite(hp->weight_decay);
  if (!ok) return fail(DOPT_E_INVALID, std::string(fn) + ": bad AdamW hyper-parameters");
  if (!std::isfinite(inv_scale)) return fail(DOPT_E_INVALID, std::string(fn) + ": bad inv_loss_scale");
  return DOPT_OK;
}

int norm_regions(int32_t n) { return std::max(1, (n + kNormCap - 1) / kNormCap); }
size_t list_workspace_bytes(int32_t n) {
  return kScalarBytes + (size_t)norm_regions(n) * kMaxGrid * sizeof(Partial);
}

int check_norm_args(int32_t n, float inv_scale, double max_norm, const void* ws, size_t bytes, const char* fn) {
  if (!std::isfinite(inv_scale) || std::isnan(max_norm))
    return fail(DOPT_E_INVALID, std::string(fn) + ": bad inv_loss_scale or max_norm");
  if (!ws) return fail(DOPT_E_INVALID, std::string(fn) + ": NULL workspace");
  if (!aligned_to(ws, 16)) return fail(DOPT_E_ALIGN, std::string(fn) + ": workspace not 16-byte aligned");
  const size_t need = list_workspace_bytes(n);
  if (bytes < need)
    return fail(DOPT_E_SIZE, std::string(fn) + ": workspace needs " + std::to_string(need) + " bytes, got " +
                                 std::to_string(bytes));
  return DOPT_OK;
}

// The 4-byte device scalars of a call (any may be NULL).
int check_scalars(const float* norm, const float* coef, const int32_t* found, const char* fn) {
  if (aligned_to(norm, 4) && aligned_to(coef, 4) && aligned_to(found, 4)) return DOPT_OK;
  return fail(DOPT_E_ALIGN, std::string(fn) + ": a norm, clip coefficient or found_inf not 4-byte aligned");
}

char* ws_at(void* ws, size_t offset) { return static_cast<char*>(ws) + offset; }

// A table's record of tiles outside their tensor (debug builds).
template <typename P>
int set_record(P& p) {
#if DOPT_BOUNDS_CHECK
  return bounds_record(&p.record);
#else
  (void)p;
  return DOPT_OK;
#endif
}

// The norm launches of a list, then the finalize.
int run_norm(const dopt_tensor* ts, int32_t n, float inv_scale, FinalizeArgs fin, void* ws, cudaStream_t s) {
  Partial* parts = reinterpret_cast<Partial*>(ws_at(ws, kScalarBytes));
  NormParamsT<kNormCap> p;
  if (int st = set_record(p)) return st;
  p.inv_scale = inv_scale;
  p.n_seg = p.n_tiles = 0;
  p.err_flag = fin.err_flag = reinterpret_cast<int32_t*>(ws_at(ws, kErrorFlagOffset));
  fin.parts = parts;
  fin.n_slots = 0;
  int32_t k = 0;
  do {
    for (; k < n && p.n_seg < kNormCap; ++k) {
      if (ts[k].numel == 0) continue;
      const size_t elem = dtype_bytes(ts[k].grad_dtype);
      const int16_t shift = (int16_t)((reinterpret_cast<uintptr_t>(ts[k].grad) & (kNormVector - 1)) / elem);
      p.seg[p.n_seg++] = NormSeg{ts[k].grad, ts[k].numel, p.n_tiles, (int16_t)ts[k].grad_dtype, shift};
      p.n_tiles += (int32_t)tiles_of(ts[k].numel + shift, tensors_norm_tile_bytes() / (int)elem);
    }
    int grid = 0;
    int st = tensors_norm_grid(p, &grid);
    if (st) return st;
    p.partials = parts + fin.n_slots;
    fin.n_slots += grid;
    if ((st = launch_tensors_norm(p, s))) return st;
    p.n_seg = p.n_tiles = 0;
  } while (k < n);
  return launch_tensors_finalize(fin, s);
}

// AdamSeg::shift of a tensor with fp32 moments: its first element's index
// within groups of 32 elements (a warp's accesses then cover whole 128-byte
// lines: 3.4 % on a list of tensors at odd elements), or of the four that
// its arrays are read in, when they agree -- as separate allocations do, and
// views of buffers at one element offset; else -1.
int32_t common_shift(const AdamSeg& g) {
  auto index = [](const void* p, size_t elem, int32_t group) {
    return (int32_t)(reinterpret_cast<uintptr_t>(p) / elem & (group - 1));
  };
  for (int32_t group : {32, 4}) {
    const int32_t at = index(g.weight, 4, group);
    if (index(g.m, 4, group) == at && index(g.v, 4, group) == at &&
        index(g.grad, dtype_bytes(g.grad_dtype), group) == at && index(g.param, dtype_bytes(g.param_dtype), group) == at)
      return at;
  }
  return -1;
}

// Whether a tensor with 8-bit moments has its first element on a vector
// boundary of every array (16 bytes, 32 for the weights): the blocks start there.
bool block_vectors(const AdamSeg& g) {
  return aligned_to(g.weight, 32) && aligned_to(g.m, 16) && aligned_to(g.v, 16) &&
         aligned_to(g.grad, 16) && aligned_to(g.param, 8 * dtype_bytes(g.param_dtype));
}

struct AdamJob {
  const dopt_adamw_hparams* hp;
  float inv_scale;
  uint32_t seed;
  const float* coef;
  const int32_t* found;
  const DevStep* dev = nullptr;
  const int64_t* d_step = nullptr;
  bool early = false;  // the launch before is this call's norm
};

// The AdamW launches of a list: one per moments' format in it (more when it
// has more tensors than a table holds).
int run_adamw(const dopt_tensor* ts, int32_t n, const AdamJob& j, cudaStream_t s) {
  const dopt_adamw_hparams* hp = j.hp;
  AdamParamsT<kAdamCap> p;
  if (int st = set_record(p)) return st;
  p.coef = j.coef;
  p.found_inf = j.found;
  p.dev = j.dev;
  p.d_step = j.d_step;
  p.lr_wd = hp->lr * hp->weight_decay;
  p.b1 = (float)hp->beta1;
  p.b2 = (float)hp->beta2;
  p.omb1 = (float)(1.0 - hp->beta1);
  p.omb2 = (float)(1.0 - hp->beta2);
  p.eps = (float)hp->eps;
  p.step_size = (float)(hp->lr / (1.0 - pow_int(hp->beta1, hp->step)));
  p.bc2_sqrt = (float)std::sqrt(1.0 - pow_int(hp->beta2, hp->step));
  p.inv_scale = j.inv_scale;
  p.key = j.seed + (j.dev ? 0u : (uint32_t)hp->step * kHashStep);
  p.early = j.early ? 1 : 0;
  for (int32_t moments : {DOPT_MOMENTS_F32, DOPT_MOMENTS_8BIT}) {
    p.n_seg = p.n_tiles = 0;
    auto flush = [&]() -> int {
      if (!p.n_seg) return DOPT_OK;
      int st = moments == DOPT_MOMENTS_F32 ? launch_tensors_adamw(p, s) : launch_tensors_adamw8(p, s);
      p.n_seg = p.n_tiles = 0;
      p.early = 1;
      return st;
    };
    for (int32_t k = 0; k < n; ++k) {
      const dopt_tensor& t = ts[k];
      if (t.numel == 0 || t.moments != moments) continue;
      if (p.n_seg == kAdamCap)
        if (int st = flush()) return st;
      AdamSeg& g = p.seg[p.n_seg++];
      g.param = t.param;
      g.grad = t.grad;
      g.weight = t.param_dtype == DOPT_F32 ? static_cast<float*>(t.param) : t.master;
      g.m = t.exp_avg;
      g.v = t.exp_avg_sq;
      g.m_scale = t.exp_avg_scale;
      g.v_scale = t.exp_avg_sq_scale;
      g.len = t.numel;
      if (j.dev)
        g.wd_mult = t.wd_mult;
      else
        g.decay = (float)(1.0 - p.lr_wd * t.wd_mult);
      g.tile0 = p.n_tiles;
      g.key = (uint32_t)k * kHashTensor;
      g.param_dtype = (int16_t)t.param_dtype;
      g.grad_dtype = (int16_t)t.grad_dtype;
      if (moments == DOPT_MOMENTS_F32) {
        g.shift = common_shift(g);
        p.n_tiles += (int32_t)tiles_of(t.numel + std::max(g.shift, 0), kAdamTile32);
      } else {
        g.shift = block_vectors(g) ? 0 : -1;
        p.n_tiles += (int32_t)tiles_of(t.numel, kAdamTile);
      }
    }
    if (int st = flush()) return st;
  }
  return DOPT_OK;
}

int check_moments(const dopt_moment_tensor* ts, int32_t n, const char* fn) {
  int st = check_list(ts, n, fn);
  if (st) return st;
  int64_t tiles = 0;
  for (int32_t k = 0; k < n; ++k) {
    const dopt_moment_tensor& t = ts[k];
    if (t.numel < 0) return fail(DOPT_E_INVALID, at(fn, k) + "negative numel");
    if (t.values_dtype != DOPT_F32 && t.values_dtype != DOPT_BF16)
      return fail(DOPT_E_INVALID, at(fn, k) + "values are fp32 or bf16");
    if (t.numel == 0) continue;
    if (!count_tiles(t.numel, &tiles)) return fail(DOPT_E_SIZE, at(fn, k) + "too many elements in the list");
    const size_t elem = dtype_bytes(t.values_dtype);
    if (t.exp_avg) {
      if ((st = check_array(t.exp_avg, elem, "exp_avg", k, fn))) return st;
      if (!t.exp_avg_codes || !t.exp_avg_scale) return fail(DOPT_E_INVALID, at(fn, k) + "NULL exp_avg codes or scales");
    }
    if (t.exp_avg_sq) {
      if ((st = check_array(t.exp_avg_sq, elem, "exp_avg_sq", k, fn))) return st;
      if (!t.exp_avg_sq_codes || !t.exp_avg_sq_scale)
        return fail(DOPT_E_INVALID, at(fn, k) + "NULL exp_avg_sq codes or scales");
    }
  }
  return DOPT_OK;
}

int run_moments(const dopt_moment_tensor* ts, int32_t n, bool pack, cudaStream_t s) {
  MomentParamsT<kMomentCap> p;
  if (int st = set_record(p)) return st;
  for (int32_t dt : {DOPT_F32, DOPT_BF16}) {
    p.n_seg = p.n_tiles = 0;
    auto flush = [&]() -> int {
      if (!p.n_seg) return DOPT_OK;
      int st = pack ? launch_state8_pack(dt, p, s) : launch_state8_unpack(dt, p, s);
      p.n_seg = p.n_tiles = 0;
      return st;
    };
    for (int32_t k = 0; k < n; ++k) {
      const dopt_moment_tensor& t = ts[k];
      if (t.numel == 0 || t.values_dtype != dt || (!t.exp_avg && !t.exp_avg_sq)) continue;
      if (p.n_seg == kMomentCap)
        if (int st = flush()) return st;
      const bool vec = (!t.exp_avg || (aligned_to(t.exp_avg, 32) && aligned_to(t.exp_avg_codes, 16))) &&
                       (!t.exp_avg_sq || (aligned_to(t.exp_avg_sq, 32) && aligned_to(t.exp_avg_sq_codes, 16)));
      p.seg[p.n_seg++] = MomentSeg{t.exp_avg,          t.exp_avg_sq,    t.exp_avg_codes,    t.exp_avg_sq_codes,
                                   t.exp_avg_scale,    t.exp_avg_sq_scale, t.numel,         p.n_tiles, vec ? 1 : 0};
      p.n_tiles += (int32_t)tiles_of(t.numel, pack ? kAdamTile : kUnpackTile);
    }
    if (int st = flush()) return st;
  }
  return DOPT_OK;
}

// Runs an entry point's body: a host allocation that fails (an error
// message's, say) is a status, not an exception through the C boundary.
template <typename F>
int guarded(const char* fn, F&& body) noexcept {
  try {
    return body();
  } catch (const std::bad_alloc&) {
    return DOPT_E_NOMEM;
  } catch (...) {
    return DOPT_E_INVALID;
  }
}

}  // namespace

extern "C" {

int64_t dopt_moment_blocks(int64_t numel) {
  return guarded("dopt_moment_blocks", [&] { return numel < 0 ? fail(DOPT_E_INVALID, "dopt_moment_blocks: negative numel") : 0; })
             ? DOPT_E_INVALID
             : numel / kMomentBlock + (numel % kMomentBlock != 0);
}

size_t dopt_tensors_workspace_bytes(int32_t n_tensors) {
  if (guarded("dopt_tensors_workspace_bytes", [&] { return check_list(&n_tensors, n_tensors, "dopt_tensors_workspace_bytes"); }))
    return 0;
  return list_workspace_bytes(n_tensors);
}

int dopt_tensors_grad_norm(const dopt_tensor* tensors, int32_t n_tensors, float inv_loss_scale, double max_norm,
                           void* workspace, size_t workspace_bytes, float* d_norm, float* d_clip_coef,
                           int32_t* d_found_inf, dopt_stream stream) {
  const char* fn = "dopt_tensors_grad_norm";
  return guarded(fn, [&]() -> int {
    int st = check_grads(tensors, n_tensors, fn);
    if (st) return st;
    if ((st = check_norm_args(n_tensors, inv_loss_scale, max_norm, workspace, workspace_bytes, fn))) return st;
    if ((st = check_scalars(d_norm, d_clip_coef, d_found_inf, fn))) return st;
    FinalizeArgs f{};
    f.max_norm = max_norm;
    f.sc = static_cast<Scalars*>(workspace);
    f.d_norm = d_norm;
    f.d_coef = d_clip_coef;
    f.d_found = d_found_inf;
    return run_norm(tensors, n_tensors, inv_loss_scale, f, workspace, (cudaStream_t)stream);
  });
}

int dopt_tensors_adam_step(const dopt_tensor* tensors, int32_t n_tensors, const dopt_adamw_hparams* hp,
                           float inv_loss_scale, uint32_t seed, const float* d_clip_coef, const int32_t* d_found_inf,
                           dopt_stream stream) {
  const char* fn = "dopt_tensors_adam_step";
  return guarded(fn, [&]() -> int {
    int st = check_states(tensors, n_tensors, fn);
    if (st) return st;
    if ((st = check_hp(hp, false, inv_loss_scale, fn))) return st;
    if ((st = check_scalars(nullptr, d_clip_coef, d_found_inf, fn))) return st;
    AdamJob j{hp, inv_loss_scale, seed, d_clip_coef, d_found_inf};
    return run_adamw(tensors, n_tensors, j, (cudaStream_t)stream);
  });
}

int dopt_tensors_step(const dopt_tensor* tensors, int32_t n_tensors, const dopt_adamw_hparams* hp,
                      float inv_loss_scale, double max_norm, uint32_t seed, int64_t* d_step, const double* d_lr,
                      void* workspace, size_t workspace_bytes, int32_t* d_found_inf, float* d_norm,
                      dopt_stream stream) {
  const char* fn = "dopt_tensors_step";
  return guarded(fn, [&]() -> int {
    int st = check_states(tensors, n_tensors, fn);
    if (st) return st;
    if ((st = check_hp(hp, d_step != nullptr, inv_loss_scale, fn))) return st;
    if ((st = check_norm_args(n_tensors, inv_loss_scale, max_norm, workspace, workspace_bytes, fn))) return st;
    if ((st = check_scalars(d_norm, nullptr, d_found_inf, fn))) return st;
    if (!aligned_to(d_step, 8) || !aligned_to(d_lr, 8))
      return fail(DOPT_E_ALIGN, std::string(fn) + ": d_step / d_lr not 8-byte aligned");
    FinalizeArgs f{};
    Scalars* sc = static_cast<Scalars*>(workspace);
    f.max_norm = max_norm;
    f.sc = sc;
    f.d_norm = d_norm;
    f.d_found = d_found_inf;
    DevStep* dev = reinterpret_cast<DevStep*>(ws_at(workspace, kDevStepOffset));
    if (d_step)
      f.step = K2Step{d_step, d_lr, hp->lr, hp->weight_decay, hp->beta1, hp->beta2, dev};
    if ((st = run_norm(tensors, n_tensors, inv_loss_scale, f, workspace, (cudaStream_t)stream))) return st;
    AdamJob j{hp, inv_loss_scale, seed, &sc->clip_coef, &sc->found_inf};
    j.dev = d_step ? dev : nullptr;
    j.d_step = d_step;
    j.early = true;
    return run_adamw(tensors, n_tensors, j, (cudaStream_t)stream);
  });
}

int dopt_state8_pack(const dopt_moment_tensor* tensors, int32_t n_tensors, dopt_stream stream) {
  const char* fn = "dopt_state8_pack";
  return guarded(fn, [&]() -> int {
    int st = check_moments(tensors, n_tensors, fn);
    return st ? st : run_moments(tensors, n_tensors, true, (cudaStream_t)stream);
  });
}

int dopt_state8_unpack(const dopt_moment_tensor* tensors, int32_t n_tensors, dopt_stream stream) {
  const char* fn = "dopt_state8_unpack";
  return guarded(fn, [&]() -> int {
    int st = check_moments(tensors, n_tensors, fn);
    return st ? st : run_moments(tensors, n_tensors, false, (cudaStream_t)stream);
  });
}

}  // extern "C"
