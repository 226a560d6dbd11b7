// matrix8_multiply_pair.cu -- products of 8-bit matrices in tiles of two SMs.
//
// Two CTAs of a cluster multiply 256 n by 256 m together: each loads its half
// of the rows of both operands, and the unit of each reads the other's half
// of a too.  Per step along k a CTA loads 32 KB for as many products as a
// single CTA's 128 x 256 tile makes of 48 KB, which is what the L2 has to
// give.  Each CTA has the sums of its 128 n.  Measured on 16384 x 11008 x 4096
// to bf16: 365 us, 4.04 PFLOP/s, with constant codes at 2070 MHz; 495 to 515
// with random ones, where the power limit holds the clock at 1400 to 1480 MHz
// (tiles of one SM, 128 x 256: 577).
#include "matrix8_mma.cuh"

namespace dopt {

struct PairShape {
  static constexpr int kTile = 256, kHalf = 128;       // n and m of a tile; rows that a CTA loads
  static constexpr int kOperand = kHalf * kOperandRow;  // bytes, of either
  static constexpr int kScaleTiles = 3;                 // of 512 bytes per stage: own rows of b, all of a's
  static constexpr int kStages = 6;
  static constexpr int kScaleAt = kStages * 2 * kOperand;
  static constexpr int kBarAt = kScaleAt + kStages * kScaleTiles * 512;
  static constexpr int kBytes = kBarAt + (2 * kStages + 2) * 8 + 16;
  static constexpr size_t kSmem = kBytes + 1024;
  // Two sets of sums, used in turn, share 32 columns: the next products may
  // start when those have been read, and the rest is read under them.
  static constexpr int kTmem = 512, kShared = 32, kSecond = kTile - kShared;
  static constexpr int kScaleCol = kSecond + kTile, kScaleCols = 4 * kScaleTiles;  // two sets, used in turn
  static_assert(kScaleCol + 2 * kScaleCols <= kTmem, "TMEM columns");
};

// An arrival on a barrier of the cluster's first CTA, from either.  It says
// that TMEM has been read, which the fence before it orders; releasing memory
// too would wait for the thread's stores of the last tile (1600 cycles).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The wait for a barrier that the other CTA's threads arrive on.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, unsigned parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, "
      "p;\n}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, unsigned parity) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  for (;;) {
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait_cluster(bar, parity)) return true;
    if (global_ns() - t0 > kWaitNs) return false;
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kMulThreads)
    matrix8_multiply_pair(const __grid_constant__ MulParams p) {
  using S = PairShape;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kBarAt);  // the first CTA's: both halves are there
  uint64_t* empty = full + S::kStages;
  uint64_t* sums = empty + S::kStages;
  uint64_t* taken = sums + 1;  // the first CTA's: in both epilogues' registers
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(taken + 1);
  volatile uint32_t* failed = tmem_at + 1;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rank = (int)(blockIdx.x & 1u);

  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    mbar_init(sums, 1);
    mbar_init(taken, 16);
    *failed = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) tmem_alloc<2>(tmem_at, S::kTmem);
  if (threadIdx.x == 96) {
    prefetch_map(&p.b_map);
    prefetch_map(&p.a_map);
    prefetch_map(&p.b_scales);
    prefetch_map(&p.a_scales);
  }
  tmem_fence_before();
  __syncthreads();
  cluster_sync();
  tmem_fence_after();
  const uint32_t tmem = *tmem_at;
  const int first = (int)(blockIdx.x >> 1), stride = (int)(gridDim.x >> 1);

  if (warp == 0) {
    if (elect_one()) {
      int stage = 0, phase = 0;
      uint32_t loads = 0;
      bool ok = true;
      for (int t = first; t < p.n_tiles && ok; t += stride) {
        const MulTile tile = mul_tile(p, t);
        for (int k = 0; k < p.blocks; ++k) {
          if (!(ok = mbar_wait_bounded(empty + stage, phase ^ 1))) break;
          uint8_t* b = smem + stage * 2 * S::kOperand;
          const bool scales = k % 4 == 0;
          // the first CTA's barrier counts both CTAs' bytes
          if (rank == 0)
            mbar_arrive_expect_tx(full + stage, 4 * S::kOperand + (scales ? 2 * 512 * S::kScaleTiles : 0));
          const uint32_t bar = cluster_addr(smem_addr(full + stage), 0);
          tma_load_2d<2>(b, &p.b_map, k * kOperandRow, tile.n * S::kTile + rank * S::kHalf, bar);
          tma_load_2d<2>(b + S::kOperand, &p.a_map, k * kOperandRow, tile.m * S::kTile + rank * S::kHalf, bar);
          if (scales) {
            uint8_t* s = smem + S::kScaleAt + stage * S::kScaleTiles * 512;
            tma_load_2d<2>(s, &p.b_scales, 0, (tile.n * 2 + rank) * p.groups + k / 4, bar);
            tma_load_2d<2>(s + 512, &p.a_scales, 0, tile.m * 2 * p.groups + k / 4, bar);
            tma_load_2d<2>(s + 1024, &p.a_scales, 0, (tile.m * 2 + 1) * p.groups + k / 4, bar);
          }
          ++loads;
          if (++stage == S::kStages) stage = 0, phase ^= 1;
        }
      }
      // no copy is in flight when the CTAs end, whoever gave up
      if (rank == 0)
        for (uint32_t i = loads > S::kStages ? loads - S::kStages : 0; i < loads; ++i)
          mbar_wait_cluster(full + i % S::kStages, (i / S::kStages) & 1);
    }
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    if (elect_one()) {
      int stage = 0, phase = 0, done = 0, set = 0;
      bool ok = true;
      for (int t = first; t < p.n_tiles && ok; t += stride) {
        for (int part = 0; part < p.blocks && ok; part += p.part, ++done) {
          if (!(ok = mbar_wait_cluster(taken, (done & 1) ^ 1))) {
            *failed = 1u;
            break;
          }
          tmem_fence_after();
          const int end = min(p.blocks, part + p.part);
          const uint32_t acc = tmem + (done & 1 ? S::kSecond : 0);
          for (int k = part; k < end; ++k) {
            if (!(ok = mbar_wait_cluster(full + stage, phase))) break;
            tmem_fence_after();
            const uint32_t b = smem_addr(smem + stage * 2 * S::kOperand);
            if (k % 4 == 0) {
              set ^= 1;
              const uint32_t s = smem_addr(smem + S::kScaleAt + stage * S::kScaleTiles * 512);
#pragma unroll
              for (int i = 0; i < S::kScaleTiles; ++i)
                scale_to_tmem<2>(tmem + S::kScaleCol + set * S::kScaleCols + 4 * i, scales_desc(s + 512 * i));
            }
            const uint32_t sb = tmem + S::kScaleCol + set * S::kScaleCols, sa = sb + 4;
            const uint32_t instr = scaled_instr(S::kTile, S::kTile) | scale_byte(k & 3);
            const uint64_t bd = operand_desc(b), ad = operand_desc(b + S::kOperand);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_scaled<2>(acc, bd + 2 * j, ad + 2 * j, instr, sb, sa, (k > part || j > 0) ? 1u : 0u);
            mma_commit<2>(empty + stage);
            if (++stage == S::kStages) stage = 0, phase ^= 1;
          }
          if (!ok) {
            *failed = 1u;
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(smem_addr(tmem_at + 1), 1)), "r"(1) : "memory");
          }
          mma_commit<2>(sums);  // after what was issued, all of a part's products or not
        }
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    constexpr int kColumns = S::kTile / 2;
    const int quarter = warp % 4, half = (warp - 4) / 4;
    const uint32_t taken_by = cluster_addr(smem_addr(taken), 0);
    bool ok = true;
    int done = 0;
    for (int t = first; t < p.n_tiles; t += stride) {
      const MulTile tile = mul_tile(p, t);
      uint32_t r[kColumns];
      for (int part = 0; part < p.blocks; part += p.part, ++done) {
        ok = ok && mbar_wait_bounded(sums, done & 1) && !*failed;
        ok = __all_sync(0xFFFFFFFFu, ok);
        tmem_fence_after();
        const uint32_t from = tmem + ((uint32_t)quarter << 21) + (done & 1 ? S::kSecond : 0) + half * kColumns;
        auto release = [&] {
          tmem_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(taken_by);
          __syncwarp();  // loads from TMEM follow
        };
        // the columns that the other set shares first: the last of the first
        // set, the first of the second
        if (done & 1) {
          if (half == 0) take_range<0, S::kShared>(from, part == 0, r);
          release();
          if (half == 1) take_range<0, S::kShared>(from, part == 0, r);
          take_range<S::kShared, kColumns>(from, part == 0, r);
        } else {
          if (half == 1) take_range<kColumns - S::kShared, kColumns>(from, part == 0, r);
          release();
          if (half == 0) take_range<kColumns - S::kShared, kColumns>(from, part == 0, r);
          take_range<0, kColumns - S::kShared>(from, part == 0, r);
        }
      }
      if (!ok) {
#pragma unroll
        for (int c = 0; c < kColumns; ++c) r[c] = 0x7FC00000u;
      }
      store_column(p, r, (int64_t)tile.n * S::kTile + rank * S::kHalf + quarter * 32 + lane,
                   (int64_t)tile.m * S::kTile + half * kColumns);
    }
  }
  tmem_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA's memory is used by the other any more
  tmem_fence_after();
  if (warp == 2) tmem_free<2>(tmem, S::kTmem);
}

int launch_multiply_pair(MulParams& p, const dopt_matrix8& a, const dopt_matrix8& b, cudaStream_t s) {
  const char* what = "matrix8_multiply_pair launch";
  using S = PairShape;
  static std::atomic<uint64_t> allowed{0};
  int st = allow_dynamic_smem(matrix8_multiply_pair, S::kSmem, allowed, what);
  if (st) return st;
  if ((st = operand_map(&p.b_map, b, S::kHalf))) return st;
  if ((st = operand_map(&p.a_map, a, S::kHalf))) return st;
  if ((st = scales_map(&p.b_scales, b)) || (st = scales_map(&p.a_scales, a))) return st;
  int sms = 0;
  if ((st = device_sms(&sms))) return st;
  p.tiles_m = (int32_t)((a.rows + S::kTile - 1) / S::kTile);
  p.tiles_n = (int32_t)((b.rows + S::kTile - 1) / S::kTile);
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  if (tiles > INT32_MAX / 8) return fail(DOPT_E_SIZE, "dopt_matrix8_multiply: too many elements in d");
  p.n_tiles = (int32_t)tiles;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min(p.n_tiles, sms / 2) * 2);
  cfg.blockDim = dim3(kMulThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, matrix8_multiply_pair, p);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(DOPT_E_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
  }
  return check_launch(what);
}

}  // namespace dopt
