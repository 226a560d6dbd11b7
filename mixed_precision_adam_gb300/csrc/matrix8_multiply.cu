// matrix8_multiply.cu -- products of 8-bit matrices, d = a b^T (+ d), in
// tiles of one SM, and the choice among the kernels.
//
// A CTA has a tile of 128 n by BT m: one warp loads 128 bytes of k of both
// operands per step by TMA into a ring, one thread issues the products, and
// eight warps take the sums from TMEM to registers at once, give TMEM back
// and store while the next tile is being multiplied.  Few rows of a are bound
// by b's bytes from HBM and by latency: 16 x 11008 x 4096 takes 11.7 us, 3.9
// TB/s, 16 x 4096 x 1024 4.4, of which 2.5 are a launch.
#include "matrix8_mma.cuh"

namespace dopt {

constexpr int kTileN = 128;

// BT: rows of a per tile.  Stages of the ring: as many as leave room for two
// CTAs per SM up to 64 rows, else for one.  A CTA's part of TMEM is no larger
// than its part of the shared memory (or it is alone on its SM), so no CTA of
// these kernels waits for TMEM that another one of a waiting cluster holds.
template <int BT>
struct MulShape {
  static constexpr int kScaleTiles = 1 + (BT + 127) / 128;  // of 512 bytes, per stage
  static constexpr int kB = kTileN * kOperandRow, kA = BT * kOperandRow;
  static constexpr int kStages = BT <= 32 ? 5 : BT == 64 ? 4 : 6;
  static constexpr int kScaleAt = kStages * (kA + kB);
  static constexpr int kBarAt = kScaleAt + kStages * kScaleTiles * 512;
  static constexpr int kBytes = kBarAt + (2 * kStages + 2) * 8 + 16;
  static constexpr size_t kSmem = kBytes + 1024;  // the ring starts on 1024 bytes
  static constexpr int kTmem = BT <= 64 ? 128 : 256;  // columns
  static constexpr int kScaleCol = BT;  // first column of the scales: two sets, used in turn
  static constexpr int kScaleCols = 4 * kScaleTiles;
  static_assert(kScaleCol + 2 * kScaleCols <= kTmem, "TMEM columns");
  static_assert(kB % 1024 == 0 && (BT < 8 || kA % 1024 == 0), "operand tiles start on an atom");
};

template <int BT, bool SPLIT>
__global__ void __launch_bounds__(kMulThreads, BT <= 64 ? 2 : 1) matrix8_multiply(const __grid_constant__ MulParams p) {
  using S = MulShape<BT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBarAt);
  uint64_t* empty = full + S::kStages;
  uint64_t* sums = empty + S::kStages;   // the tile's sums are complete
  uint64_t* taken = sums + 1;            // and in the epilogue's registers
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(taken + 1);
  volatile uint32_t* failed = tmem_at + 1;  // a wait ran out
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    mbar_init(sums, 1);
    mbar_init(taken, 8);
    *failed = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) tmem_alloc<1>(tmem_at, S::kTmem);
  if (threadIdx.x == 96) {
    prefetch_map(&p.b_map);
    prefetch_map(&p.a_map);
    prefetch_map(&p.b_scales);
    prefetch_map(&p.a_scales);
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = *tmem_at;

  // this CTA's tiles and its share of k, in groups of four blocks
  int first = blockIdx.x, stride = gridDim.x, rank = 0;
  int k0 = 0, k1 = p.blocks;
  if constexpr (SPLIT) {
    rank = (int)(blockIdx.x & ((1u << p.split_log) - 1u));
    first = (int)(blockIdx.x >> p.split_log);
    stride = p.n_tiles;  // one tile
    k0 = p.groups * rank >> p.split_log << 2;  // groups < 2^22
    k1 = min(p.blocks, p.groups * (rank + 1) >> p.split_log << 2);
  }

  if (warp == 0) {
    if (elect_one()) {
      int stage = 0, phase = 0;
      uint32_t loads = 0;
      bool ok = true;
      for (int t = first; t < p.n_tiles && ok; t += stride) {
        const MulTile tile = mul_tile(p, t);
        for (int k = k0; k < k1; ++k) {
          if (!(ok = mbar_wait_bounded(empty + stage, phase ^ 1))) break;
          uint8_t* b = smem + stage * (S::kA + S::kB);
          uint8_t* a = b + S::kB;
          const bool scales = k % 4 == 0;
          const uint32_t bar = smem_addr(full + stage);
          mbar_arrive_expect_tx(full + stage, S::kA + S::kB + (scales ? 512 * S::kScaleTiles : 0));
          tma_load_2d<1>(b, &p.b_map, k * kOperandRow, tile.n * kTileN, bar);
          tma_load_2d<1>(a, &p.a_map, k * kOperandRow, tile.m * BT, bar);
          if (scales) {
            uint8_t* s = smem + S::kScaleAt + stage * S::kScaleTiles * 512;
            tma_load_2d<1>(s, &p.b_scales, 0, tile.n * p.groups + k / 4, bar);
#pragma unroll
            for (int i = 1; i < S::kScaleTiles; ++i)
              tma_load_2d<1>(s + 512 * i, &p.a_scales, 0, (tile.m * BT / 128 + i - 1) * p.groups + k / 4, bar);
          }
          ++loads;
          if (++stage == S::kStages) stage = 0, phase ^= 1;
        }
      }
      // no copy is in flight when the CTA ends, whoever gave up
      for (uint32_t i = loads > S::kStages ? loads - S::kStages : 0; i < loads; ++i)
        mbar_wait_bounded(full + i % S::kStages, (i / S::kStages) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      int stage = 0, phase = 0, done = 0, set = 0;
      bool ok = true;
      for (int t = first; t < p.n_tiles && ok; t += stride) {
        for (int part = k0; part < k1 && ok; part += p.part, ++done) {
          if (!(ok = mbar_wait_bounded(taken, (done & 1) ^ 1))) {
            *failed = 1u;
            break;
          }
          tmem_fence_after();
          const int end = min(k1, part + p.part);
          for (int k = part; k < end; ++k) {
            if (!(ok = mbar_wait_bounded(full + stage, phase))) break;
            tmem_fence_after();
            const uint32_t b = smem_addr(smem + stage * (S::kA + S::kB)), a = b + S::kB;
            if (k % 4 == 0) {
              set ^= 1;
              const uint32_t s = smem_addr(smem + S::kScaleAt + stage * S::kScaleTiles * 512);
#pragma unroll
              for (int i = 0; i < S::kScaleTiles; ++i)
                scale_to_tmem<1>(tmem + S::kScaleCol + set * S::kScaleCols + 4 * i, scales_desc(s + 512 * i));
            }
            const uint32_t sb = tmem + S::kScaleCol + set * S::kScaleCols, sa = sb + 4;
            const uint32_t instr = scaled_instr(kTileN, BT) | scale_byte(k & 3);
            const uint64_t bd = operand_desc(b), ad = operand_desc(a);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_scaled<1>(tmem, bd + 2 * j, ad + 2 * j, instr, sb, sa, (k > part || j > 0) ? 1u : 0u);
            mma_commit<1>(empty + stage);
            if (++stage == S::kStages) stage = 0, phase ^= 1;
          }
          if (!ok) *failed = 1u;
          mma_commit<1>(sums);  // after what was issued, all of a part's products or not
        }
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    constexpr int kColumns = BT / 2;
    const int quarter = warp % 4, half = (warp - 4) / 4;
    bool ok = true;
    int done = 0;
    for (int t = first; t < p.n_tiles; t += stride) {
      const MulTile tile = mul_tile(p, t);
      uint32_t r[kColumns];
      for (int part = k0; part < k1; part += p.part, ++done) {
        ok = ok && mbar_wait_bounded(sums, done & 1) && !*failed;
        ok = __all_sync(0xFFFFFFFFu, ok);
        tmem_fence_after();
        take_sums(tmem + ((uint32_t)quarter << 21) + half * kColumns, part == k0, r);
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(taken);
        __syncwarp();
      }
      if (!ok) {
#pragma unroll
        for (int c = 0; c < kColumns; ++c) r[c] = 0x7FC00000u;
      }
      if constexpr (SPLIT) {
        // a CTA leaves its sums in its own shared memory, which no copy and no
        // product uses any more; then each of the cluster adds up a share of
        // the tile's columns, in the CTAs' order
        float* mine = reinterpret_cast<float*>(smem) + quarter * 32 + lane;
#pragma unroll
        for (int c = 0; c < kColumns; ++c) mine[(half * kColumns + c) * 128] = __uint_as_float(r[c]);
        if (!ok) *failed = 1u;  // a copy of a CTA that gave up may still land on its sums
        cluster_sync();
        uint32_t bad = 0u;
        for (int q = 0; q < 1 << p.split_log; ++q) bad |= cluster_word(cluster_addr(smem_addr(tmem_at + 1), q));
        const int share = 1 << p.share_log, ctas = 1 << p.split_log;
        for (int c = warp - 4; c < share; c += 8) {
          const int64_t row = (int64_t)tile.m * BT + rank * share + c, n = (int64_t)tile.n * kTileN + lane * 4;
          if (row >= p.m) break;
          const uint32_t at = smem_addr(smem) + (uint32_t)(rank * share + c) * 512u + (uint32_t)lane * 16u;
          float4 sum = cluster_load(cluster_addr(at, 0));
#pragma unroll
          for (int q0 = 1; q0 < 8; q0 += 4) {
            float4 x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (q0 + j < ctas) x[j] = cluster_load(cluster_addr(at, q0 + j));
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (q0 + j < ctas) sum = make_float4(sum.x + x[j].x, sum.y + x[j].y, sum.z + x[j].z, sum.w + x[j].w);
          }
          if (n >= p.n) continue;
          if (bad) sum.x = sum.y = sum.z = sum.w = __int_as_float(0x7FC00000);
          if (p.dtype == DOPT_F32)
            store_four<float>(p, sum, n, row);
          else if (p.dtype == DOPT_BF16)
            store_four<__nv_bfloat16>(p, sum, n, row);
          else
            store_four<__half>(p, sum, n, row);
        }
        cluster_sync();  // the others have read what lies here
      } else {
        store_column(p, r, (int64_t)tile.n * kTileN + quarter * 32 + lane, (int64_t)tile.m * BT + half * kColumns);
      }
    }
  }
  if constexpr (SPLIT) {
    if (warp < 4) {
      cluster_sync();
      cluster_sync();
    }
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == 2) tmem_free<1>(tmem, S::kTmem);
}

// --------------------------------------------------------------------- host --

namespace {
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder of tensor maps, looked up once.
int tensor_map_encoder(EncodeTiled* out) {
  static std::atomic<void*> known{nullptr};
  void* f = known.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult q;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q);
    if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !f) {
      (void)cudaGetLastError();
      return fail(DOPT_E_CUDA, "cuTensorMapEncodeTiled is not available");
    }
    known.store(f, std::memory_order_release);
  }
  *out = reinterpret_cast<EncodeTiled>(f);
  return DOPT_OK;
}

}  // namespace

int operand_map(CUtensorMap* map, const dopt_matrix8& m, int box) {
  EncodeTiled encode;
  if (int st = tensor_map_encoder(&encode)) return st;
  const cuuint64_t size[2] = {(cuuint64_t)m.cols, (cuuint64_t)m.rows}, stride[1] = {(cuuint64_t)m.ld};
  const cuuint32_t tile[2] = {kOperandRow, (cuuint32_t)box}, step[2] = {1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, m.codes, size, stride, tile, step,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DOPT_OK : fail(DOPT_E_CUDA, "cuTensorMapEncodeTiled failed: " + std::to_string((int)r));
}

int scales_map(CUtensorMap* map, const dopt_matrix8& m) {
  EncodeTiled encode;
  if (int st = tensor_map_encoder(&encode)) return st;
  const cuuint64_t size[2] = {128, (cuuint64_t)(scale_size(m.rows, m.cols) / 512)}, stride[1] = {512};
  const cuuint32_t tile[2] = {128, 1}, step[2] = {1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, m.scales, size, stride, tile, step,
                            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DOPT_OK : fail(DOPT_E_CUDA, "cuTensorMapEncodeTiled failed: " + std::to_string((int)r));
}

namespace {

template <int BT, bool SPLIT>
int launch_multiply(MulParams& p, const dopt_matrix8& a, const dopt_matrix8& b, cudaStream_t s) {
  const char* what = "matrix8_multiply launch";
  using S = MulShape<BT>;
  static std::atomic<uint64_t> allowed{0};
  auto kern = matrix8_multiply<BT, SPLIT>;
  int st = allow_dynamic_smem(kern, S::kSmem, allowed, what);
  if (st) return st;
  if ((st = operand_map(&p.b_map, b, kTileN))) return st;
  if ((st = operand_map(&p.a_map, a, BT))) return st;
  if ((st = scales_map(&p.b_scales, b)) || (st = scales_map(&p.a_scales, a))) return st;
  int sms = 0;
  if ((st = device_sms(&sms))) return st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = SPLIT ? 1u << p.split_log : 1u;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(SPLIT ? p.n_tiles << p.split_log : std::min(p.n_tiles, sms * (BT <= 64 ? 2 : 1))));
  cfg.blockDim = dim3(kMulThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(DOPT_E_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
  }
  return check_launch(what);
}

// What a product takes, in units of 10 ns, by fits to 3 x 11 x 4 sizes of k, m
// and n (bf16, weights not in L2): a launch, and for each wave of tiles its
// steps along k and its start and end.
struct Plan {
  int64_t cost;
  int split_log;
};
int64_t waves_of(int64_t tiles, int64_t at_once) { return (tiles + at_once - 1) / at_once; }
int64_t pair_cost(int64_t m, int64_t n, int64_t blocks, int sms) {
  return 650 + waves_of((m + 255) / 256 * ((n + 255) / 256), sms / 2) * (blocks * 26 + 200);
}
// Tiles of one SM, their k split over a cluster of CTAs where that leaves
// none of them to a second wave and is worth its exchange: 128 x 2048 x 4096
// takes 7.9 us split in four and 10.2 whole, 128 x 2048 x 1024 7.5 and 5.4.
// Clusters of eight need eight free SMs of one GPC each, so they are left to
// few tiles (128 x 2048 x 4096 in eight: 12.9 us).
Plan one_sm_plan(int bt, int64_t tiles, int64_t blocks, int64_t groups, int sms) {
  const int64_t slots = sms * (bt <= 64 ? 2 : 1);
  static const int exchange[2][4] = {{0, 120, 140, 150}, {0, 270, 270, 270}};
  Plan best{410 + waves_of(tiles, slots) * (blocks * 19 + 100), 0};
  for (int s = 1; s <= 3; ++s) {
    const int64_t ctas = tiles << s;
    if (ctas > (s < 3 ? slots : bt <= 64 ? sms : sms / 2) || groups < (1 << s)) break;
    const int64_t cost = 510 + (blocks * 19 >> s) + exchange[bt > 32][s];
    if (cost < best.cost) best = Plan{cost, s};
  }
  return best;
}

template <int BT>
int multiply_rows(MulParams& p, const dopt_matrix8& a, const dopt_matrix8& b, int sms, cudaStream_t s) {
  p.tiles_m = (int32_t)((a.rows + BT - 1) / BT);
  p.tiles_n = (int32_t)((b.rows + kTileN - 1) / kTileN);
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  if (tiles > INT32_MAX / 8) return fail(DOPT_E_SIZE, "dopt_matrix8_multiply: too many elements in d");
  p.n_tiles = (int32_t)tiles;
  p.split_log = one_sm_plan(BT, tiles, p.blocks, p.groups, sms).split_log;
  p.share_log = 0;
  while ((1 << p.split_log << p.share_log) < BT) ++p.share_log;
  return p.split_log ? launch_multiply<BT, true>(p, a, b, s) : launch_multiply<BT, false>(p, a, b, s);
}

}  // namespace
}  // namespace dopt

using namespace dopt;

extern "C" int dopt_matrix8_multiply(const dopt_matrix8* a, const dopt_matrix8* b, void* d, int32_t d_dtype, int64_t ldd,
                                     int32_t accumulate, dopt_stream stream) {
  return guard_entry([&]() -> int {
    const std::string fn = "dopt_matrix8_multiply: ";
    if (!a || !b) return fail(DOPT_E_INVALID, fn + "NULL matrix");
    int st = check_sides(a->rows, a->cols, fn + "a: ");
    if (st) return st;
    if ((st = check_sides(b->rows, b->cols, fn + "b: "))) return st;
    if (a->cols != b->cols) return fail(DOPT_E_INVALID, fn + "a and b have different cols");
    if (!known_dtype(d_dtype)) return fail(DOPT_E_INVALID, fn + "unknown dtype of d");
    if (a->rows == 0 || b->rows == 0) return DOPT_OK;
    const size_t elem = dtype_bytes(d_dtype);
    if (!d) return fail(DOPT_E_INVALID, fn + "NULL d");
    if (!aligned_to(d, elem)) return fail(DOPT_E_ALIGN, fn + "d not aligned to its elements");
    if ((st = check_ld(ldd, b->rows, fn + "d: "))) return st;
    const cudaStream_t s = (cudaStream_t)stream;
    if (a->cols == 0) {
      if (accumulate) return DOPT_OK;
      return check_memset(cudaMemset2DAsync(d, (size_t)ldd * elem, 0, (size_t)b->rows * elem, (size_t)a->rows, s), fn);
    }
    if ((st = check_matrix8(*a, fn + "a: "))) return st;
    if ((st = check_matrix8(*b, fn + "b: "))) return st;
    MulParams p{};
    p.d = d;
    p.ldd = ldd;
    p.m = (int32_t)a->rows;
    p.n = (int32_t)b->rows;
    p.blocks = (int32_t)row_blocks(a->cols);
    p.groups = (int32_t)scale_groups(a->cols);
    if (scale_size(std::max(a->rows, b->rows), a->cols) / 512 > INT32_MAX / 2)
      return fail(DOPT_E_SIZE, fn + "too many elements");
    p.part = d_dtype == DOPT_F32 ? kPart : kPart16;
    p.dtype = d_dtype;
    p.accumulate = accumulate ? 1 : 0;
    const int64_t m = a->rows, n = b->rows;
    int sms = 0;
    if ((st = device_sms(&sms))) return st;
    if (m <= 16) return multiply_rows<16>(p, *a, *b, sms, s);
    if (m <= 32) return multiply_rows<32>(p, *a, *b, sms, s);
    if (m <= 64) return multiply_rows<64>(p, *a, *b, sms, s);
    const int64_t tiles = (m + 127) / 128 * ((n + kTileN - 1) / kTileN);
    if (m > 128 && pair_cost(m, n, p.blocks, sms) < one_sm_plan(128, tiles, p.blocks, p.groups, sms).cost)
      return launch_multiply_pair(p, *a, *b, s);
    return multiply_rows<128>(p, *a, *b, sms, s);
  });
}
