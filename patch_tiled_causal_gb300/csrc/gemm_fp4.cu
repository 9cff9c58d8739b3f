// Product of two microscaled 4-bit operands on the 5th-generation tensor cores (tcgen05, sm_103a):
//   D[m, n] = alpha * sum_k (a[m, k] sa[m, k / block]) (b[n, k] sb[n, k / block]) + bias[n]
// with e2m1 a, b and power-of-two (MXFP4, block 32) or e4m3 (NVFP4, block 16) scales, which the tensor cores
// apply to the products of each block before the fp32 accumulation (kind::mxf4, kind::mxf4nvf4).
//
// A k block is 256 columns: 128 bytes of codes per row, which one TMA box brings into a 128-byte-swizzled
// K-major tile, and 8 (MXFP4) or 16 (NVFP4) scale bytes per row, which arrive as whole 128-row x 4-block tiles
// of 512 bytes and go from shared into tensor memory with tcgen05.cp (32 lanes x 16 bytes, repeated for the
// four lane quadrants).  Each MMA takes 64 columns.  Rows and columns beyond the operands arrive as
// zeros, and the MMAs of the last k block stop at K, so any size works without padding.  The scales of
// stage s live in their own columns of tensor memory: the copy that overwrites them is issued after the barrier
// that says the stage's MMAs are done.
//
// Two kernels:
//   gemm_fp4_pair_kernel   persistent; a cluster of 2 CTAs runs 256 x 256 tiles as cta_group::2 MMAs, each CTA
//                          holding its 128 rows of A, half of B's rows and the scales of all of them.
//   gemm_fp4_split_kernel  few tiles: one CTA per 128 x 128 tile and part of K, the parts of a tile in one
//                          cluster, whose CTAs add the partial sums up through distributed shared memory.
#include <algorithm>
#include <cstring>
#include <mutex>

#include "common.cuh"
#include "fp4.cuh"
#include "gemm_store.cuh"
#include "internal.h"

namespace vae {

struct Fp4GemmParams {
  int M, N, K;
  int num_kb;         // k blocks of 256 columns
  int n_ntiles, n_tiles;
  int split;          // CTAs (cluster size) that share one tile's K
  float alpha;
  const float* bias;
  void* y;
  int out_f32;
  int vec;            // rows of D start on 16-byte boundaries
  int whole16;        // rows of D are whole 16-byte chunks long
  int64_t ldd;
  uint32_t* fault;
  uint64_t limit_ns;
};

namespace {

constexpr int kBlockM = 128;
constexpr int kKB = 256;                            // columns per k block
constexpr uint32_t kTileBytes = kBlockM * kKB / 2;  // codes of 128 rows
constexpr int kEpiWarps = 8;                        // two per TMEM lane quadrant, each half of the columns
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr uint32_t kTmemCols = 512;

template <int kFmt> constexpr int kGroups = kFmt == VAE_MXFP4 ? 2 : 4;  // 4-block scale groups per k block

// The issuing loop runs inside one election: per k block it issues 6 (MXFP4) or 12 (NVFP4) scale copies, 4 MMAs and a
// commit, and issuing bounds the kernel when each costs much (16384 x 4096 x 4096, MXFP4 / NVFP4, 4 stages: a loop
// under lane == 0 143 / 187 us, this way 103 / 107).
// D[tmem] (+)= A B^T with block scales in tensor memory, 64 columns of K.
#define VAE_MMA_FP4(CTA, KIND, VEC)                                                                             \
  asm volatile(                                                                                                 \
      "{\n\t.reg .pred p;\n\t"                                                                                  \
      "setp.ne.b32 p, %6, 0;\n\t"                                                                               \
      "tcgen05.mma.cta_group::" CTA ".kind::" KIND ".block_scale.scale_vec::" VEC                               \
      " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),                                                   \
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)                                 \
      : "memory")
template <int kFmt, bool kPair>
VAE_DEV void tc_mma_fp4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                        uint32_t accumulate) {
  if constexpr (kFmt == VAE_MXFP4 && kPair) VAE_MMA_FP4("2", "mxf4", "2X");
  else if constexpr (kFmt == VAE_MXFP4) VAE_MMA_FP4("1", "mxf4", "2X");
  else if constexpr (kPair) VAE_MMA_FP4("2", "mxf4nvf4", "4X");
  else VAE_MMA_FP4("1", "mxf4nvf4", "4X");
}
#undef VAE_MMA_FP4

// One 512-byte scale tile from shared into 4 columns of tensor memory (pair: in each of the two CTAs).
template <bool kPair>
VAE_DEV void tc_cp_scales(uint32_t taddr, uint64_t sdesc) {
  if constexpr (kPair) asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
  else asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

// Shared-memory descriptor of a scale tile: 32 rows of 16 bytes, no swizzle, 8-row groups 128 bytes apart.
VAE_DEV uint64_t sdesc_scales(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);  // start address
  d |= static_cast<uint64_t>(128u >> 4) << 16;           // leading byte offset (unused: one 16-byte column)
  d |= static_cast<uint64_t>(128u >> 4) << 32;           // stride byte offset
  d |= static_cast<uint64_t>(1u) << 46;                  // descriptor version
  return d;
}

// Instruction descriptor: e2m1 A and B (K-major), fp32 D, M x N; scales e8m0 (MXFP4) or e4m3; `sf_id` the byte of
// each 32-bit scale word where this MMA's scales start (MXFP4 takes 2 of the 4, NVFP4 all).
template <int kFmt>
VAE_DEV constexpr uint32_t idesc_fp4(uint32_t m, uint32_t n, uint32_t sf_id) {
  return (sf_id << 4)                                       // B scale id
         | (1u << 7) | (1u << 10)                           // A, B format: e2m1
         | ((n >> 3) << 17)                                 // N / 8
         | ((kFmt == VAE_MXFP4 ? 1u : 0u) << 23)            // scale format: e8m0 / e4m3
         | ((m >> 7) << 27)                                 // M / 128
         | (sf_id << 29);                                   // A scale id
}

// One k block in shared memory at a_addr: A codes, B codes, A scales [group], B scales [128-row tile][group];
// kBTiles: 128-row tiles of B's scales (each CTA of a pair holds all of them).  One lane calls these.
template <int kFmt, bool kPair, int kBTiles>
VAE_DEV void issue_scales(uint32_t a_addr, uint32_t sf_tmem) {
  constexpr uint32_t kG = kGroups<kFmt>;
  const uint32_t sa_addr = a_addr + 2u * kTileBytes;
  const uint32_t sb_addr = sa_addr + kG * 512u;
  const uint32_t sfb = sf_tmem + 4u * kG;
#pragma unroll
  for (uint32_t g = 0; g < kG; ++g) {
    tc_cp_scales<kPair>(sf_tmem + 4u * g, sdesc_scales(sa_addr + g * 512u));
#pragma unroll
    for (uint32_t j = 0; j < kBTiles; ++j)
      tc_cp_scales<kPair>(sfb + 4u * (g * kBTiles + j), sdesc_scales(sb_addr + (j * kG + g) * 512u));
  }
}

template <int kFmt, bool kPair, int kBTiles>
VAE_DEV void issue_mmas(uint32_t a_addr, uint32_t sf_tmem, uint32_t d_tmem, int steps, bool first) {
  constexpr uint32_t kG = kGroups<kFmt>;
  const uint32_t sfb = sf_tmem + 4u * kG;
  const uint64_t adesc = sdesc_kmajor_sw128(a_addr);
  const uint64_t bdesc = sdesc_kmajor_sw128(a_addr + kTileBytes);
  constexpr uint32_t m = kPair ? 2 * kBlockM : kBlockM, n = 128u * kBTiles;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k >= steps) break;
    const uint32_t g = kFmt == VAE_MXFP4 ? k >> 1 : k;
    const uint32_t id = kFmt == VAE_MXFP4 ? (k & 1) * 2 : 0;
    tc_mma_fp4<kFmt, kPair>(d_tmem, adesc + 2u * k, bdesc + 2u * k, idesc_fp4<kFmt>(m, n, id), sf_tmem + 4u * g,
                            sfb + 4u * kBTiles * g, (first && k == 0) ? 0u : 1u);
  }
}

}  // namespace

// ================================================================================ 256 x 256 tiles, CTA pairs
// Warp 0 loads, warp 1 (of the leader) issues, warps 2..9 drain: 8 warps read the accumulator's 128 x 256
// values of their CTA into registers and hand it back at once, then scale, add the bias, round, and store
// while the next tile's MMAs run.  One accumulator of 256 columns leaves tensor memory for the scales of 5 stages
// (two of 192 columns load more per product: 73920 x 1024 x 1024 NVFP4 52 us against 45).
// Stores: each warp lays 32 rows x 128 bytes into its own swizzled buffer and a TMA store writes it (row-wise
// 16-byte stores from the buffer: 73920 x 1024 x 256 43.6 us against 30.5); where D's rows are not 16-byte
// aligned, or N ends inside 16 bytes, the warp writes the buffer row by row (73920 x 1023 x 1024 58 us).
// 16384 x 4096 x 4096 MXFP4 takes 88 us, 73920 x 1024 x 1024 NVFP4 42.  Of the former the loads alone take 73 us
// (16 TB/s from L2) and the MMAs of K = 64 with their scale copies alone 72 us (7.6 PFLOP/s, the rate of this
// instruction and not the chip's: the form with K = 96 is not used); the two do not overlap fully.
namespace {
constexpr int kPairBN = 256;
constexpr int kPairStages = 5;
constexpr uint32_t kPairSfCol = 256;  // scales behind the accumulator
template <int kFmt> constexpr uint32_t kPairStage = 2u * kTileBytes + 3u * kGroups<kFmt> * 512u;
template <int kFmt>
constexpr uint32_t kPairSmem = kPairStages * kPairStage<kFmt> + kEpiWarps * (kStoreBuf + 512u) +
                               (2u * kPairStages + 2u) * 8u + 16u;
static_assert(kPairSmem<VAE_NVFP4> <= 227u * 1024u, "shared memory");
static_assert(kPairSfCol + kPairStages * 12u * kGroups<VAE_NVFP4> <= kTmemCols, "tensor memory");

template <typename TO>
VAE_DEV void drain_tile(const Fp4GemmParams& p, const CUtensorMap* tmD, uint8_t* buf, const float* bias_s,
                        const uint32_t* raw, int row0, int n0, int lane) {
  constexpr int kCols = 128 / static_cast<int>(sizeof(TO));
#pragma unroll
  for (int j = 0; j < 128 / kCols; ++j) {
    float v[kCols];
#pragma unroll
    for (int i = 0; i < kCols; i += 4) {
      const float4 b = *reinterpret_cast<const float4*>(bias_s + j * kCols + i);
      v[i] = fmaf(__uint_as_float(raw[j * kCols + i]), p.alpha, b.x);
      v[i + 1] = fmaf(__uint_as_float(raw[j * kCols + i + 1]), p.alpha, b.y);
      v[i + 2] = fmaf(__uint_as_float(raw[j * kCols + i + 2]), p.alpha, b.z);
      v[i + 3] = fmaf(__uint_as_float(raw[j * kCols + i + 3]), p.alpha, b.w);
    }
    if (lane == 0) bulk_wait_read();  // the previous store has read the buffer
    __syncwarp();
    store_slab<TO>(p, tmD, buf, v, row0, n0 + j * kCols, lane);
  }
}
}  // namespace

template <int kFmt>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_fp4_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                         const __grid_constant__ CUtensorMap tmD, const __grid_constant__ Fp4GemmParams p) {
  constexpr int kG = kGroups<kFmt>;
  constexpr uint32_t kStage = kPairStage<kFmt>;
  constexpr int kStages = kPairStages;
  extern __shared__ __align__(1024) uint8_t smem[];  // (128-byte-swizzled tiles: 1024-byte atoms)
  uint8_t* store_bufs = smem + kStages * kStage;
  float* bias_bufs = reinterpret_cast<float*>(store_bufs + kEpiWarps * kStoreBuf);
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(bias_bufs + kEpiWarps * 128);
  uint64_t* empty_bar = full_bar + kStages;
  uint64_t* accf_bar = empty_bar + kStages;
  uint64_t* acce_bar = accf_bar + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acce_bar + 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int tile0 = blockIdx.x >> 1, tile_step = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(accf_bar, 1);
    mbar_init(acce_bar, 2 * kEpiWarps);
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSA);
    tma_prefetch_desc(&tmSB);
    if (p.vec) tma_prefetch_desc(&tmD);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  cluster_sync();  // the peer's barriers and tensor memory exist before anything targets them

  if (warp == 0) {
    if (lane == 0) {
      int kc = 0, s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = tile0; tile < p.n_tiles && ok; tile += tile_step) {
        const int mt = tile / p.n_ntiles, nt = tile - mt * p.n_ntiles;
        for (int kb = 0; kb < p.num_kb; ++kb, ++kc) {
          if (kc >= kStages && !mbar_wait(&empty_bar[s], ph ^ 1u, p.fault, p.limit_ns, 51)) {
            ok = false;
            break;
          }
          uint8_t* a = smem + s * kStage;
          uint8_t* sa = a + 2 * kTileBytes;
          // both CTAs' tiles complete on the leader's barrier (the leader alone runs the MMAs)
          const uint32_t fb = cluster_map(smem_u32(&full_bar[s]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&full_bar[s], 2 * kStage);
          tma_load_2d_pair(a, &tmA, fb, kb * (kKB / 2), (2 * mt + rank) * kBlockM);
          tma_load_2d_pair(a + kTileBytes, &tmB, fb, kb * (kKB / 2), nt * kPairBN + rank * kBlockM);
          tma_load_3d_pair(sa, &tmSA, fb, 0, kb * kG, 2 * mt + rank);
          tma_load_3d_pair(sa + kG * 512, &tmSB, fb, 0, kb * kG, 2 * nt);
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // every load has landed and every commit has arrived before the CTA may exit
      if (rank == 0)
        for (int k = max(0, kc - kStages); k < kc; ++k)
          mbar_wait(&full_bar[k % kStages], (k / kStages) & 1, p.fault, p.limit_ns, 52);
      for (int k = max(0, kc - kStages); k < kc; ++k)
        mbar_wait(&empty_bar[k % kStages], (k / kStages) & 1, p.fault, p.limit_ns, 57);
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      const uint32_t smem_base = smem_u32(smem);
      int s = 0, it = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = tile0; tile < p.n_tiles && ok; tile += tile_step, ++it) {
        if (it > 0 && !mbar_wait(acce_bar, (it - 1) & 1, p.fault, p.limit_ns, 56)) break;
        tc_fence_after();
        for (int kb = 0; kb < p.num_kb; ++kb) {
          if (!mbar_wait(&full_bar[s], ph, p.fault, p.limit_ns, 53)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_addr = smem_base + static_cast<uint32_t>(s) * kStage;
          const uint32_t sf_tmem = tmem_base + kPairSfCol + static_cast<uint32_t>(s) * (12u * kG);
          issue_scales<kFmt, true, 2>(a_addr, sf_tmem);
          issue_mmas<kFmt, true, 2>(a_addr, sf_tmem, tmem_base, min(4, (p.K - kb * kKB + 63) / 64), kb == 0);
          tc_commit_pair_arrive_both(&empty_bar[s], 0x3);
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
        tc_commit_pair_arrive_both(accf_bar, 0x3);
      }
    }
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;  // TMEM lane quadrant this warp may access, half of the columns
    uint8_t* buf = store_bufs + (warp - 2) * kStoreBuf;
    float* bias_s = bias_bufs + (warp - 2) * 128;
    int it = 0;
    for (int tile = tile0; tile < p.n_tiles; tile += tile_step, ++it) {
      const int mt = tile / p.n_ntiles, nt = tile - mt * p.n_ntiles;
      const int row0 = (2 * mt + rank) * kBlockM + q * 32;
      const int n0 = nt * kPairBN + half * 128;
      float4 b4 = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p.bias) {
        const int n = n0 + lane * 4;
        if (n < p.N) b4.x = __ldg(p.bias + n);
        if (n + 1 < p.N) b4.y = __ldg(p.bias + n + 1);
        if (n + 2 < p.N) b4.z = __ldg(p.bias + n + 2);
        if (n + 3 < p.N) b4.w = __ldg(p.bias + n + 3);
      }
      __syncwarp();  // the previous tile's bias has been read
      reinterpret_cast<float4*>(bias_s)[lane] = b4;
      // (one answer for the warp, which the .aligned loads below want whole, also where some lanes' waits ran out)
      if (!__all_sync(0xffffffffu, mbar_wait(accf_bar, it & 1, p.fault, p.limit_ns, 55))) break;
      tc_fence_after();
      uint32_t raw[128];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        tmem_ld_32x32b_x32(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(half * 128 + j * 32),
                           raw + 32 * j);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster_relaxed(cluster_map(smem_u32(acce_bar), 0));
      if (p.out_f32) drain_tile<float>(p, &tmD, buf, bias_s, raw, row0, n0, lane);
      else drain_tile<__nv_bfloat16>(p, &tmD, buf, bias_s, raw, row0, n0, lane);
    }
    if (lane == 0) bulk_wait_read();  // the stores have left shared memory before the CTA exits
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();  // (one of its lanes comes from the issuing loop)
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
  cluster_sync();  // neither CTA leaves while the other may still write into it
}

// ================================================================================ few tiles: split K in a cluster
// One CTA per (128 x 128 tile, part of K).  Each drains its partial sums into shared memory (over the stages, which
// are done with); the CTAs of a tile's cluster then each add up and store 1 / split of the tile's rows, reading the
// other CTAs' sums through distributed shared memory in a fixed order.
namespace {
constexpr int kSplitStages = 5;
constexpr uint32_t kSplitSfCol = 128;
template <int kFmt> constexpr uint32_t kSplitStage = 2u * kTileBytes + 2u * kGroups<kFmt> * 512u;
constexpr uint32_t kSumPitch = 132;  // floats per row of partial sums: rows 16 bytes off each other's banks
template <int kFmt>
constexpr uint32_t kSplitSmem = 1024u + kSplitStages * kSplitStage<kFmt> + (2u * kSplitStages + 1u) * 8u + 16u;
static_assert(kSplitStages * kSplitStage<VAE_MXFP4> >= kBlockM * kSumPitch * 4u, "the sums lie over the stages");
static_assert(kSplitSmem<VAE_NVFP4> <= 227u * 1024u, "shared memory");
static_assert(kSplitSfCol + kSplitStages * 8u * kGroups<VAE_NVFP4> <= kTmemCols, "tensor memory");
}  // namespace

namespace {
// This CTA's rows of the tile, part, part + S, ...: the S CTAs' sums added up in order, scaled, stored; 4 columns per
// thread and item, 16 loads in flight (one row at a time the exchange cost 15 ns a row).
template <int S>
VAE_DEV void add_parts(const Fp4GemmParams& p, uint32_t sums, int part, int mt, int nt) {
  constexpr int kItems = 16 / S;
  const int rows = min(kBlockM, p.M - mt * kBlockM);
  const int items = (rows - part + S - 1) / S * 32;  // (this CTA's rows) x 32 groups of columns
  const int lane = threadIdx.x & 31;
  const int n = nt * kBlockM + lane * 4;
  float b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = p.bias && n + i < p.N ? __ldg(p.bias + n + i) : 0.f;
  uint32_t base[S];
#pragma unroll
  for (int c = 0; c < S; ++c) base[c] = cluster_map(sums, c) + lane * 16;
  for (int i0 = threadIdx.x; i0 < items; i0 += kItems * kThreads) {
    float4 u[kItems][S];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int r = part + ((i0 + k * kThreads) >> 5) * S;
      if (r < rows) {
#pragma unroll
        for (int c = 0; c < S; ++c) u[k][c] = ld_cluster_f4(base[c] + r * (kSumPitch * 4));
      }
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
      const int r = part + ((i0 + k * kThreads) >> 5) * S;
      if (r >= rows) break;
      float4 t = u[k][0];
#pragma unroll
      for (int c = 1; c < S; ++c) {
        t.x += u[k][c].x; t.y += u[k][c].y; t.z += u[k][c].z; t.w += u[k][c].w;
      }
      const float v[4] = {fmaf(t.x, p.alpha, b[0]), fmaf(t.y, p.alpha, b[1]), fmaf(t.z, p.alpha, b[2]),
                          fmaf(t.w, p.alpha, b[3])};
      const int64_t off = static_cast<int64_t>(mt * kBlockM + r) * p.ldd + n;
      if (p.vec && n + 4 <= p.N) {
        if (p.out_f32) {
          *reinterpret_cast<float4*>(static_cast<float*>(p.y) + off) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
          uint2 w;
          reinterpret_cast<__nv_bfloat162*>(&w)[0] = __floats2bfloat162_rn(v[0], v[1]);
          reinterpret_cast<__nv_bfloat162*>(&w)[1] = __floats2bfloat162_rn(v[2], v[3]);
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.y) + off) = w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < p.N) {
            if (p.out_f32) static_cast<float*>(p.y)[off + i] = v[i];
            else static_cast<__nv_bfloat16*>(p.y)[off + i] = f2bf(v[i]);
          }
      }
    }
  }
}
}  // namespace

template <int kFmt>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_fp4_split_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                          const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                          const __grid_constant__ Fp4GemmParams p) {
  constexpr int kG = kGroups<kFmt>;
  constexpr uint32_t kStage = kSplitStage<kFmt>;
  constexpr int kStages = kSplitStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + kStages * kStage);
  uint64_t* empty_bar = full_bar + kStages;
  uint64_t* accf_bar = empty_bar + kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accf_bar + 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int tile = blockIdx.x / p.split, part = blockIdx.x - tile * p.split;
  const int mt = tile / p.n_ntiles, nt = tile - mt * p.n_ntiles;
  const int kb0 = part * p.num_kb / p.split, kb1 = (part + 1) * p.num_kb / p.split;  // at least one k block

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(accf_bar, 1);
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      int kb = kb0;
      for (; kb < kb1; ++kb) {
        if (kb - kb0 >= kStages && !mbar_wait(&empty_bar[s], ph ^ 1u, p.fault, p.limit_ns, 61)) break;
        uint8_t* a = smem + s * kStage;
        uint8_t* sa = a + 2 * kTileBytes;
        mbar_arrive_expect_tx(&full_bar[s], kStage);
        tma_load_2d(a, &tmA, &full_bar[s], kb * (kKB / 2), mt * kBlockM);
        tma_load_2d(a + kTileBytes, &tmB, &full_bar[s], kb * (kKB / 2), nt * kBlockM);
        tma_load_3d(sa, &tmSA, &full_bar[s], 0, kb * kG, mt);
        tma_load_3d(sa + kG * 512, &tmSB, &full_bar[s], 0, kb * kG, nt);
        if (++s == kStages) {
          s = 0;
          ph ^= 1u;
        }
      }
      const int n = kb - kb0;  // every load has landed before its memory is used for the sums
      for (int k = max(0, n - kStages); k < n; ++k)
        mbar_wait(&full_bar[k % kStages], (k / kStages) & 1, p.fault, p.limit_ns, 62);
    }
  } else if (warp == 1) {
    const uint32_t smem_base = smem_u32(smem);
    int s = 0;
    uint32_t ph = 0;
    if (elect_one()) {
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&full_bar[s], ph, p.fault, p.limit_ns, 63)) break;
        tc_fence_after();
        const uint32_t a_addr = smem_base + static_cast<uint32_t>(s) * kStage;
        const uint32_t sf_tmem = tmem_base + kSplitSfCol + static_cast<uint32_t>(s) * (8u * kG);
        issue_scales<kFmt, false, 1>(a_addr, sf_tmem);
        issue_mmas<kFmt, false, 1>(a_addr, sf_tmem, tmem_base, min(4, (p.K - kb * kKB + 63) / 64), kb == kb0);
        tc_commit(&empty_bar[s]);
        if (++s == kStages) {
          s = 0;
          ph ^= 1u;
        }
      }
      tc_commit(accf_bar);
    }
    __syncwarp();
    mbar_wait(accf_bar, 0, p.fault, p.limit_ns, 64);
  }
  __syncthreads();  // loads landed, MMAs done (or given up on): the stages become the sums
  tc_fence_after();
  float* sums = reinterpret_cast<float*>(smem);
  if (warp >= 2) {
    const int q = warp & 3, half = (warp - 2) >> 2;
    if (mt * kBlockM + q * 32 < p.M) {
      uint32_t raw[64];
      const uint32_t t = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(half * 64);
      tmem_ld_32x32b_x32(t, raw);
      tmem_ld_32x32b_x32(t + 32u, raw + 32);
      tmem_ld_wait();
      float* dst = sums + (q * 32 + lane) * kSumPitch + half * 64;
#pragma unroll
      for (int i = 0; i < 64; i += 4)
        *reinterpret_cast<float4*>(dst + i) = make_float4(__uint_as_float(raw[i]), __uint_as_float(raw[i + 1]),
                                                          __uint_as_float(raw[i + 2]), __uint_as_float(raw[i + 3]));
    }
    tc_fence_before();
  }
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
  switch (p.split) {
    case 8: add_parts<8>(p, smem_u32(sums), part, mt, nt); break;
    case 4: add_parts<4>(p, smem_u32(sums), part, mt, nt); break;
    case 2: add_parts<2>(p, smem_u32(sums), part, mt, nt); break;
    default: add_parts<1>(p, smem_u32(sums), part, mt, nt); break;
  }
  cluster_sync();  // no CTA leaves while another may still read its sums
}

// ================================================================================ host side
namespace {
std::mutex g_mu;
struct DevInfo {
  bool ready = false;
  int n_sm = 0;
  int clusters[2] = {0, 0};          // pairs resident at once, by format
  int split_clusters[3] = {0, 0, 0};  // clusters of 2, 4, 8 CTAs of the split kernel resident at once
};
DevInfo g_dev[64];

cudaLaunchConfig_t cluster_config(cudaLaunchAttribute* attr, unsigned grid, unsigned cluster, size_t smem,
                                  cudaStream_t stream) {
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = cluster;
  attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

cudaError_t device_info(DevInfo* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lk(g_mu);
  DevInfo& d = g_dev[dev];
  if (!d.ready) {
    e = cudaDeviceGetAttribute(&d.n_sm, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    for (auto* k : {gemm_fp4_split_kernel<VAE_MXFP4>, gemm_fp4_split_kernel<VAE_NVFP4>}) {
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
      if (e != cudaSuccess) return e;
    }
    int i = 0;
    for (auto* k : {gemm_fp4_pair_kernel<VAE_MXFP4>, gemm_fp4_pair_kernel<VAE_NVFP4>}) {
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
      if (e != cudaSuccess) return e;
      cudaLaunchAttribute attr;
      cudaLaunchConfig_t cfg = cluster_config(&attr, 2 * (d.n_sm / 2), 2, i ? kPairSmem<VAE_NVFP4> : kPairSmem<VAE_MXFP4>, nullptr);
      int mc = 0;
      if (cudaOccupancyMaxActiveClusters(&mc, k, &cfg) != cudaSuccess || mc <= 0) mc = d.n_sm / 2;
      d.clusters[i++] = mc;
    }
    for (int k = 0; k < 3; ++k) {  // (NVFP4, the larger of the two in shared memory)
      cudaLaunchAttribute attr;
      cudaLaunchConfig_t cfg = cluster_config(&attr, 2u << k, 2u << k, kSplitSmem<VAE_NVFP4>, nullptr);
      int mc = 0;
      if (cudaOccupancyMaxActiveClusters(&mc, gemm_fp4_split_kernel<VAE_NVFP4>, &cfg) != cudaSuccess) mc = 0;
      d.split_clusters[k] = mc;
    }
    d.ready = true;
  }
  *out = d;
  return cudaSuccess;
}
}  // namespace

cudaError_t launch_gemm_fp4(const Fp4GemmArgs& a, cudaStream_t stream) {
  DevInfo dev;
  cudaError_t e = device_info(&dev);
  if (e != cudaSuccess) return e;
  const bool mx = a.format == VAE_MXFP4;
  Fp4GemmParams p{};
  p.M = a.M; p.N = a.N; p.K = a.K;
  p.num_kb = (a.K + kKB - 1) / kKB;
  p.alpha = a.alpha; p.bias = a.bias; p.y = a.y; p.out_f32 = a.out_f32; p.ldd = a.ldd;
  p.vec = (reinterpret_cast<uintptr_t>(a.y) & 15) == 0 && (a.ldd * (a.out_f32 ? 4 : 2)) % 16 == 0;
  p.whole16 = (static_cast<int64_t>(a.N) * (a.out_f32 ? 4 : 2)) % 16 == 0;
  p.fault = fault_word();
  p.limit_ns = wait_limit_ns();

  const uint64_t pitch = static_cast<uint64_t>(a.K + 31) / 32 * 16;
  const uint64_t groups = static_cast<uint64_t>(fp4_groups(a.format, a.K));
  const uint32_t kg = mx ? kGroups<VAE_MXFP4> : kGroups<VAE_NVFP4>;
  const auto code_map = [&](CUtensorMap* m, const void* base, int rows) {
    const uint64_t dims[2] = {pitch, static_cast<uint64_t>(rows)};
    const uint64_t strides[1] = {pitch};
    const uint32_t box[2] = {kKB / 2, kBlockM};
    return make_map(m, base, 2, dims, strides, box, 1);
  };
  const auto scale_map = [&](CUtensorMap* m, const void* base, int rows, uint32_t box_tiles) {
    const uint64_t dims[3] = {128, groups, (static_cast<uint64_t>(rows) + 127) / 128};
    const uint64_t strides[2] = {512, 512 * groups};
    const uint32_t box[3] = {128, kg, box_tiles};
    return make_map(m, base, 3, dims, strides, box, 4, false);
  };
  const int64_t tiles128 = ((static_cast<int64_t>(a.M) + 127) / 128) * ((static_cast<int64_t>(a.N) + 127) / 128);
  // 128 x 128 tiles that fit the machine in one wave run in the split kernel, K in as many parts (1, 2, 4 or 8, a k block
  // or more each) as still all run at once.  Pair kernel against split, NVFP4: 1 x 1024 x 1024 5.8 us against 4.1 (4
  // parts), 1 x 1024 x 4096 9.3 against 4.7 (8), 2048 x 1024 x 1024 (128 tiles) 6.8 against 6.6 (1); 256 tiles, two
  // waves of the split kernel, 6.8 against 14.  Clusters that do not all fit at once double the time.
  const bool split = tiles128 <= dev.n_sm;
  int parts = 1;
  for (int k = 2; k >= 0 && parts == 1; --k)
    if (tiles128 <= dev.split_clusters[k] && (2 << k) <= p.num_kb) parts = 2 << k;
  CUtensorMap tmA, tmB, tmSA, tmSB, tmD;
  memset(&tmD, 0, sizeof(tmD));
  if (!code_map(&tmA, a.a_codes, a.M) || !code_map(&tmB, a.b_codes, a.N) || !scale_map(&tmSA, a.a_scales, a.M, 1) ||
      !scale_map(&tmSB, a.b_scales, a.N, split ? 1 : 2))
    return cudaErrorInvalidValue;
  cudaLaunchAttribute attr;
  if (split) {
    p.n_ntiles = (a.N + 127) / 128;
    p.n_tiles = static_cast<int>(tiles128);
    p.split = parts;
    cudaLaunchConfig_t cfg = cluster_config(&attr, static_cast<unsigned>(p.n_tiles * p.split), p.split,
                                            mx ? kSplitSmem<VAE_MXFP4> : kSplitSmem<VAE_NVFP4>, stream);
    return cudaLaunchKernelEx(&cfg, mx ? gemm_fp4_split_kernel<VAE_MXFP4> : gemm_fp4_split_kernel<VAE_NVFP4>, tmA, tmB,
                              tmSA, tmSB, p);
  }
  p.n_ntiles = (a.N + kPairBN - 1) / kPairBN;
  const int64_t tiles = (static_cast<int64_t>(a.M) + 255) / 256 * p.n_ntiles;
  if (tiles > 0x40000000LL) return cudaErrorInvalidValue;  // (refused by the entry point)
  p.n_tiles = static_cast<int>(tiles);
  p.split = 1;
  if (p.vec) {
    const uint64_t esz = a.out_f32 ? 4 : 2;
    const uint64_t dims[2] = {static_cast<uint64_t>(a.N), static_cast<uint64_t>(a.M)};
    const uint64_t strides[1] = {static_cast<uint64_t>(a.ldd) * esz};
    const uint32_t box[2] = {static_cast<uint32_t>(128 / esz), 32};
    if (!make_map(&tmD, a.y, 2, dims, strides, box, static_cast<int>(esz))) return cudaErrorInvalidValue;
  }
  const unsigned clusters = static_cast<unsigned>(std::min<int64_t>(tiles, dev.clusters[mx ? 0 : 1]));
  cudaLaunchConfig_t cfg = cluster_config(&attr, 2 * clusters, 2, mx ? kPairSmem<VAE_MXFP4> : kPairSmem<VAE_NVFP4>, stream);
  return cudaLaunchKernelEx(&cfg, mx ? gemm_fp4_pair_kernel<VAE_MXFP4> : gemm_fp4_pair_kernel<VAE_NVFP4>, tmA, tmB, tmSA,
                            tmSB, tmD, p);
}

}  // namespace vae
