// matrix8_mma.cuh -- what the products' kernels share: the PTX forms of the
// tensor cores, their memory and the copies that feed them, descriptors, the
// parameters, and the way of the sums from TMEM to d.
//   matrix8_multiply.cu      -- tiles of one SM; the C entry point
//   matrix8_multiply_pair.cu -- tiles of two
//
// The 5th-generation tensor cores multiply e4m3 codes and apply one scale
// byte per row and 32 of k themselves (kind::mxf8f6f4, block_scale): a block
// of 128 columns is four such steps with the same byte.  The bytes lie in
// memory as the unit wants them in TMEM, so they are copied, never unpacked.
//
// The unit's rows ("lanes" of TMEM) are b's rows and its columns are a's: a
// thread then holds one output column n for many m, and a warp's stores of
// one m are 32 consecutive elements, whatever the row distance or alignment
// of d.
#pragma once

#include <cuda.h>

#include "matrix8.cuh"
#include "tma.cuh"

namespace dopt {

// ---------------------------------------------------------------- PTX forms --

__device__ __forceinline__ bool elect_one() {
  uint32_t pred;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(pred));
  return pred != 0;
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// A box to this CTA's shared memory; with CTAS 2 the barrier (an address of
// the cluster's) may be the other CTA's.
template <int CTAS>
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if constexpr (CTAS == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// The address in the cluster of what CTA `rank` has at a shared address.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t at, uint32_t rank) {
  uint32_t out;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(out) : "r"(at), "r"(rank));
  return out;
}
__device__ __forceinline__ uint32_t cluster_word(uint32_t at) {
  uint32_t x;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
  return x;
}
__device__ __forceinline__ float4 cluster_load(uint32_t at) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(at) : "memory");
  return x;
}
// A cluster's barrier.  It, like the loads from TMEM, wants the lanes of a
// warp together, which they need not be after a branch of their own.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
template <int CTAS>
__device__ __forceinline__ void tmem_alloc(uint32_t* at, uint32_t columns) {
  if constexpr (CTAS == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(at)), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(at)), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
}
template <int CTAS>
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t columns) {
  if constexpr (CTAS == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns));
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns));
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// The products issued so far arrive on a barrier when they are done; with
// CTAS 2 on both CTAs' barriers.
template <int CTAS>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  if constexpr (CTAS == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"((uint16_t)3)
        : "memory");
}
// 512 scale bytes (32 x 16) to four TMEM columns, in all four lane quarters;
// with CTAS 2 in both CTAs, each from its own shared memory.
template <int CTAS>
__device__ __forceinline__ void scale_to_tmem(uint32_t tmem, uint64_t desc) {
  if constexpr (CTAS == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}
template <int CTAS>
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t instr, uint32_t sa, uint32_t sb,
                                           uint32_t add) {
  if constexpr (CTAS == 1)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(instr), "r"(sa), "r"(sb), "r"(add)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(instr), "r"(sa), "r"(sb), "r"(add)
        : "memory");
}
// N consecutive columns of the warp's 32 lanes.
template <int N>
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t* r);
template <>
__device__ __forceinline__ void tmem_load<8>(uint32_t at, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(at));
}
template <>
__device__ __forceinline__ void tmem_load<16>(uint32_t at, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at));
}

// -------------------------------------------------------------- descriptors --

// An operand's tile in shared memory: rows of 128 bytes in the 128-byte
// swizzle, eight rows to an atom of 1024 bytes; a step of 32 bytes along k
// starts 32 bytes on in the first row.
__device__ __forceinline__ uint64_t operand_desc(uint32_t smem) {
  return (uint64_t)((smem & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
         (uint64_t)2 << 61;
}
// 32 rows of 16 scale bytes, no swizzle: eight rows to 128 bytes.
__device__ __forceinline__ uint64_t scales_desc(uint32_t smem) {
  return (uint64_t)((smem & 0x3FFFFu) >> 4) | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}
// e4m3 both (0), scale bytes as powers of two (bit 23), both operands along
// k, `rows` by n columns; which byte of a scale column is per product.
__host__ __device__ constexpr uint32_t scaled_instr(int rows, int n) {
  return (uint32_t)(n >> 3) << 17 | 1u << 23 | (uint32_t)(rows >> 4) << 24;
}
__device__ __forceinline__ uint32_t scale_byte(uint32_t k) { return k << 4 | k << 29; }

// --------------------------------------------------------------- parameters --

struct MulParams {
  CUtensorMap b_map, a_map;          // codes
  CUtensorMap b_scales, a_scales;    // scale bytes, 512 at a time
  void* d;
  int64_t ldd;
  int32_t m, n;            // rows of a, of b
  int32_t blocks, groups;  // of k: 128 columns, 512 columns
  int32_t tiles_n, tiles_m, n_tiles;
  int32_t split_log, share_log;  // log2 of the CTAs of a cluster that share a tile's k, and of the rows of a that each then stores
  int32_t part;   // blocks that the matrix unit adds up before its sums are added in registers
  int32_t dtype, accumulate;
};

constexpr int kMulThreads = 384;  // load, multiply, TMEM, idle; eight warps of the epilogue
constexpr int kOperandRow = 128;  // bytes of k per step

// A tile's place: tiles are taken in bands of eight along n, so that the
// CTAs at work share rows of both operands in L2.
struct MulTile {
  int n, m;
};
constexpr int kBand = 8;
__device__ __forceinline__ MulTile mul_tile(const MulParams& p, int t) {
  const int per_band = kBand * p.tiles_m, band = t / per_band, in = t - band * per_band;
  const int width = min(kBand, p.tiles_n - band * kBand);
  return MulTile{band * kBand + in % width, in / width};
}

// One column n of d for N consecutive m, `count` of them there: rounded once,
// with what d holds added before.  fp32 sums are added where d is kept (every
// element once, so in a fixed order): a load would be waited for, and with it
// the next tile's sums (11008 x 4096 x 16384 added to fp32: 444 us so).
template <typename T, int N>
__device__ __forceinline__ void store_sums(const uint32_t (&r)[N], T* d, int64_t ldd, int count, bool accumulate) {
  if constexpr (sizeof(T) == 4) {
    if (accumulate) {
#pragma unroll
      for (int c = 0; c < N; ++c)
        if (c < count) atomicAdd(d + c * ldd, __uint_as_float(r[c]));
      return;
    }
  }
  constexpr int kAhead = N < 8 ? N : 8;  // loads under way
#pragma unroll
  for (int c = 0; c < N; c += kAhead) {
    float old[kAhead];
    if (accumulate) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) old[j] = c + j < count ? widen<T>(d[(c + j) * ldd]) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      float x = __uint_as_float(r[c + j]);
      if (accumulate) x += old[j];
      if (c + j < count) d[(c + j) * ldd] = narrow<T>(x);
    }
  }
}

// Columns C0 to C1 of a warp's share of the sums, from TMEM column `at` on,
// into r: stored at the first part of k, added at the later ones.
template <int C0, int C1, int N>
__device__ __forceinline__ void take_range(uint32_t at, bool first, uint32_t (&r)[N]) {
  constexpr int kChunk = N < 16 ? N : 16;
  if (first) {
#pragma unroll
    for (int c = C0; c < C1; c += kChunk) tmem_load<kChunk>(at + c, r + c);
    tmem_wait_load();
  } else {
#pragma unroll
    for (int c = C0; c < C1; c += kChunk) {
      uint32_t t[kChunk];
      tmem_load<kChunk>(at + c, t);
      tmem_wait_load();
#pragma unroll
      for (int j = 0; j < kChunk; ++j)
        r[c + j] = __float_as_uint(__uint_as_float(r[c + j]) + __uint_as_float(t[j]));
    }
  }
}
template <int N>
__device__ __forceinline__ void take_sums(uint32_t at, bool first, uint32_t (&r)[N]) {
  take_range<0, N>(at, first, r);
}
// The column n of d that a thread has sums of, from row m0 on.
template <int N>
__device__ __forceinline__ void store_column(const MulParams& p, const uint32_t (&r)[N], int64_t n, int64_t m0) {
  if (n >= p.n) return;
  const int count = (int)min((int64_t)N, p.m - m0);
  const int64_t at = m0 * p.ldd + n;
  if (p.dtype == DOPT_F32)
    store_sums(r, static_cast<float*>(p.d) + at, p.ldd, count, p.accumulate);
  else if (p.dtype == DOPT_BF16)
    store_sums(r, static_cast<__nv_bfloat16*>(p.d) + at, p.ldd, count, p.accumulate);
  else
    store_sums(r, static_cast<__half*>(p.d) + at, p.ldd, count, p.accumulate);
}

// Four consecutive columns n of a row m of d, those that are there.
template <typename T>
__device__ __forceinline__ void store_four(const MulParams& p, float4 x, int64_t n, int64_t m) {
  T* d = static_cast<T*>(p.d) + m * p.ldd + n;
  const int count = (int)min((int64_t)4, p.n - n);
  const float f[4] = {x.x, x.y, x.z, x.w};
  if (!p.accumulate && count == 4 && (reinterpret_cast<uintptr_t>(d) & (4 * sizeof(T) - 1)) == 0) {
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float4*>(d) = x;
    else
      *reinterpret_cast<uint2*>(d) = make_uint2(narrow_pair<T>(make_float2(x.x, x.y)), narrow_pair<T>(make_float2(x.z, x.w)));
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t one[1] = {__float_as_uint(f[j])};
    if (j < count) store_sums(one, d + j, p.ldd, 1, p.accumulate);
  }
}

// The matrix unit's sums in fp32 do not round to nearest: over a long k they
// drift, by 3e-6 of the result at 16384 and in proportion.  For fp32 results
// it adds up kPart blocks at a time and the parts are added in registers
// (11008 x 4096 x 16384: an error of 7e-7 for 3e-6, and 2 % of the time);
// kPart16 for 16-bit results, so that no wait for a part grows with k.
constexpr int kPart = 32, kPart16 = 1024;

// Products of pairs of SMs; see matrix8_multiply_pair.cu.
int launch_multiply_pair(MulParams& p, const dopt_matrix8& a, const dopt_matrix8& b, cudaStream_t s);

// The driver's maps of a matrix: codes in boxes of 128 bytes by `box` rows
// (what lies outside reads as 0), and scale bytes.
int operand_map(CUtensorMap* map, const dopt_matrix8& m, int box);
int scales_map(CUtensorMap* map, const dopt_matrix8& m);

}  // namespace dopt
