// Product of two 8-bit operands with block scales on the 5th-generation tensor cores (tcgen05, sm_103a):
//   D[m, n] = alpha * sum_kb sa[kb, m] sb[kb, n / 128] * (sum over the 128 columns k of kb of a[m, k] b[n, k]) + bias[n]
// with e4m3 a, b (kind::f8f6f4, fp32 accumulation) and fp32 scales, which no tensor core instruction takes: each k block
// goes into an accumulator of its own in tensor memory, and while the next k block multiplies, warps read it, scale it
// and add it to sums in fp32 registers.
//
// A k block is 128 columns: 128 bytes per row, which one TMA box brings into a 128-byte-swizzled K-major tile.  Rows
// and columns beyond the operands arrive as zeros, so any size works without padding.
//
// Two kernels:
//   gemm_fp8_pair_kernel   persistent; a cluster of 2 CTAs runs 256 x 256 tiles as cta_group::2 MMAs, each CTA holding
//                          its 128 rows of A and half of B's rows; two accumulators of 256 columns fill tensor memory.
//   gemm_fp8_split_kernel  few tiles or few rows of A: up to 64 rows of A as the MMA's columns and 128 rows of B as its
//                          rows, or tiles of 128 x 128; one CTA per tile and part of K, the parts of a tile in one
//                          cluster, whose CTAs add the partial sums up through distributed shared memory.
#include <algorithm>
#include <cstring>
#include <mutex>

#include "common.cuh"
#include "fp8.cuh"
#include "gemm_store.cuh"
#include "internal.h"

namespace vae {

struct Fp8GemmParams {
  int M, N, K;
  int num_kb;         // k blocks of 128 columns
  int n_ntiles, n_tiles;
  int split;          // CTAs (cluster size) that share one tile's K
  int nb;             // row blocks of B (scales per k block)
  float alpha;
  const float* sa;    // [num_kb][M]
  const float* sb;    // [num_kb][nb]
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
constexpr int kKB = 128;                        // columns (and bytes) per k block
constexpr uint32_t kTileBytes = kBlockM * kKB;  // codes of 128 rows

// A k block's sums are multiplied by the product of two scales a, b, which may leave fp32's range at either end where the
// result does not: the sums lie between 2^-18 and 448^2 * 128.  Such scales (wide_scales) multiply as two factors, the first
// of them in tensor memory (tmem_scale).  Infinities, NaN and zeros multiply as they are, and so does a scale of 2^-126, the least
// that quantisation writes (blocks of zeros have it): an error of at most 2^-150 * 448^2 * 128 < 2^-125 for each k block.
constexpr float kMinNormal = 0x1p-126f, kMaxFinite = 3.402823466e38f;
VAE_DEV bool in_range(float s) { return (fabsf(s) >= kMinNormal) & (fabsf(s) <= kMaxFinite); }
VAE_DEV float one_for_least(float a) { return fabsf(a) == kMinNormal ? 1.0f : a; }
VAE_DEV bool wide_scales(float a, float b) {
  const float x = fabsf(a), y = fabsf(b);
  const bool numbers = (x > 0.f) & (x <= kMaxFinite) & (y > 0.f) & (y <= kMaxFinite);
  return numbers & !in_range(one_for_least(a) * one_for_least(b));
}
// sum * a b = (sum * first) * second.  Sums of zero stay zero; a factor cut off at the largest finite number stands for
// results of 2^237 and above, a subnormal one for results below 2^-227.
VAE_DEV void scale_factors(float a, float b, float& first, float& second) {
  first = 1.0f;
  second = a * b;
  if (!wide_scales(a, b)) return;
  if (fabsf(second) >= 1.0f) {  // past the top: both are 1 or more
    first = fminf(fmaxf((a * 0x1p-64f) * (b * 0x1p-63f), -kMaxFinite), kMaxFinite);
    second = 0x1p127f;
  } else {  // both are below 2^23
    first = (a * 0x1p63f) * (b * 0x1p63f);
    second = 0x1p-126f;
  }
}

// Waits for this thread's tensor memory loads; v: the registers they fill, which nothing may use before.
VAE_DEV void tmem_wait_x32(uint32_t* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13])
               :
               : "memory");
  asm volatile(""
               : "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]),
                 "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                 "+r"(v[30]), "+r"(v[31])
               :
               : "memory");
}

VAE_DEV void tmem_wait_x16(uint32_t* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13])
               :
               : "memory");
  asm volatile("" : "+r"(v[14]), "+r"(v[15]) : : "memory");
}
VAE_DEV void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 "
      "[%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
// kCols columns of this warp's lanes of an accumulator times factor(column), in place: the way of wide scales, whose adds then
// are the others'.  (Small and out of their way: the multiplications between the adds, in registers, make every call's
// k blocks slower, 16384 x 4096 x 4096 223 us.)
template <int kCols, typename F>
VAE_DEV void tmem_scale(uint32_t taddr, F factor) {
#pragma unroll 1
  for (int c = 0; c < kCols; c += 16) {
    uint32_t r[16];
    tmem_ld_32x32b_x16(taddr + c, r);
    tmem_wait_x16(r);
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * factor(c + i));
    tmem_st_32x32b_x16(taddr + c, r);
  }
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// The same for columns whose scales are a0 of lane c (columns below 32) or a1 of lane c - 32, and b; the second factors of
// this lane's columns.  (A call keeps it out of the loop's registers.)
template <int kCols>
__device__ __noinline__ float2 tmem_scale_columns(uint32_t taddr, float a0, float a1, float b) {
  float f0, f1 = 1.f, s0, s1 = 1.f;
  scale_factors(a0, b, f0, s0);
  if constexpr (kCols > 32) scale_factors(a1, b, f1, s1);
  tmem_scale<kCols>(taddr, [&](int c) { return __shfl_sync(0xffffffffu, c < 32 ? f0 : f1, c % 32); });
  return make_float2(s0, s1);
}

// Whether a phase is complete (address in shared memory).
VAE_DEV bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// 4 bytes from global to shared memory while the thread goes on (cp.async.wait_all); zero where there are none.
VAE_DEV void copy4_async(uint32_t to, const float* from, bool there) {
  if (there) asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
  else asm volatile("st.shared.f32 [%0], %1;" ::"r"(to), "f"(0.f) : "memory");
}
VAE_DEV float lds_f32(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

VAE_DEV uint32_t lds_u32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// mbar_arrive_cluster_relaxed in the lanes that `yes` holds for, without a branch
VAE_DEV void arrive_if(bool yes, uint32_t bar_cluster) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar_cluster),
      "r"(static_cast<uint32_t>(yes))
      : "memory");
}

// Whether three phases are complete, asked for together (addresses in shared memory): on the issuing thread each round
// trip counts, about 100 cycles of the 512 that a k block's products take.
VAE_DEV bool mbar_try_three(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t b2, uint32_t p12) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q, r;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 q, [%3], %5;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 r, [%4], %5;\n\t"
      "and.pred p, p, q;\n\t"
      "and.pred p, p, r;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(b0), "r"(p0), "r"(b1), "r"(b2), "r"(p12)
      : "memory");
  return ok != 0;
}

// D[tmem] = A B^T over a k block of 128 columns: four MMAs of 32, from the low words of the tiles' descriptors.
VAE_DEV void mma_kblock_pair(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc) {
#pragma unroll
  for (uint32_t k = 0; k < 4; ++k)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %3};\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %4, p;\n\t}" ::"r"(d),
        "r"(a_lo + 2u * k), "r"(b_lo + 2u * k), "r"(hi), "r"(idesc), "r"(k)
        : "memory");
}
VAE_DEV void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

VAE_DEV F2 f2_bits(uint32_t lo, uint32_t hi) { return f2(__uint_as_float(lo), __uint_as_float(hi)); }

}  // namespace

// ================================================================================ 256 x 256 tiles, CTA pairs
// Warp 0 loads, warp 1 (of the leader) issues, half of the columns after half, warps 2 and 3 bring the scales of the coming
// k blocks, 4 at a time, into a ring in shared memory, already multiplied, warps 4..11 add up: two per tensor memory
// lane quadrant, one for each half, they hold the tile's 128 x 256 sums of their CTA in registers (128 a thread).  The
// first 4 warps hand registers over to them.
//
// What bounds it is the way of an accumulator there and back: MMAs and their completion seen by the adding warps (about 960
// cycles from issue), read and added up to the release (400), the release of the slower CTA seen by the issuing
// thread (500); tensor memory holds two k blocks of 256 x 256, so a k block takes about 900 cycles, where its MMAs take 512
// and its operands' way from L2 650.  16384 x 4096 x 4096 takes 201 us, 2.7 PFLOP/s (in a long stream of such calls 222: at the
// power limit the clock falls from 2.07 to 1.8 GHz); without the hand-over 147, with it but nothing read 171.
// On the way (us): all 256 columns handed over at once 247; each barrier asked for on its own by the issuing thread 246 (that thread alone then takes 670 cycles a k block); the next accumulator asked for before
// the last adds 231 -> 223, and its first reads issued between them 207 (with the warp's number uniform to the compiler, which
// frees registers); two store buffers for one and four stages for five 202.  Slower: 16 adding warps of 64 columns 243;
// one CTA's MMAs by itself with B's tile multicast 278; 96 columns read at a time 323 (spills).
namespace {
constexpr int kPairEpi = 8;
constexpr int kPairThreads = 32 * (4 + kPairEpi);
// registers a thread: 168 at launch (384 threads), then 56 for 4 warps and 224 for 8: 56 + 2 * 224 = 3 * 168
constexpr int kRegsLaunch = 168, kRegsHelp = 56, kRegsAdd = 224;
static_assert(kRegsHelp + 2 * kRegsAdd <= 3 * kRegsLaunch, "registers");
constexpr int kPairBN = 256;
constexpr int kPairStages = 4;  // (5, with one store buffer a warp: 73920 x 1024 x 1024 85.8 us, this way 82.5)
constexpr int kHalf = kPairBN / 2;  // columns (rows of B) of a half: an accumulator, and a block of B's scales
constexpr uint32_t kPairStage = 2u * kTileBytes;
constexpr int kGroup = 4;                             // k blocks whose scales come at once; the ring holds two groups
constexpr uint32_t kRing = 2u * kGroup * 2u * 128u;  // floats: [k block][half of the columns][row]
constexpr uint32_t kPairSmem = kPairStages * kPairStage + kPairEpi * (2u * kStoreBuf + 512u) + 2u * kRing * 4u +
                               (2u * kPairStages + 12u) * 8u + 32u;
static_assert(kPairSmem <= 227u * 1024u, "shared memory");

VAE_DEV void bulk_wait_read_but_one() { asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory"); }

// acc += s * (32 columns of the accumulator)
VAE_DEV void add_scaled(F2* acc, const uint32_t* raw, F2 s) {
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = f2_fma(f2_bits(raw[2 * i], raw[2 * i + 1]), s, acc[i]);
}

template <typename TO>
VAE_DEV void store_sums(const Fp8GemmParams& p, const CUtensorMap* tmD, uint8_t* buf, const float* bias_s, const F2* acc,
                        int row0, int n0, int lane) {
  constexpr int kCols = 128 / static_cast<int>(sizeof(TO));
#pragma unroll
  for (int j = 0; j < 128 / kCols; ++j) {
    float v[kCols];
#pragma unroll
    for (int i = 0; i < kCols; i += 4) {
      const float4 b = *reinterpret_cast<const float4*>(bias_s + j * kCols + i);
      const float2 t = f2_get(acc[(j * kCols + i) / 2]), u = f2_get(acc[(j * kCols + i) / 2 + 1]);
      v[i] = fmaf(t.x, p.alpha, b.x);
      v[i + 1] = fmaf(t.y, p.alpha, b.y);
      v[i + 2] = fmaf(u.x, p.alpha, b.z);
      v[i + 3] = fmaf(u.y, p.alpha, b.w);
    }
    if (lane == 0) bulk_wait_read_but_one();  // the store before the last has read its buffer, this one's
    __syncwarp();
    store_slab<TO>(p, tmD, buf + (j & 1) * kStoreBuf, v, row0, n0 + j * kCols, lane);
  }
}
}  // namespace

__global__ void __launch_bounds__(kPairThreads, 1)
    gemm_fp8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ CUtensorMap tmD, const __grid_constant__ Fp8GemmParams p) {
  constexpr int kStages = kPairStages;
  extern __shared__ __align__(1024) uint8_t smem[];  // (128-byte-swizzled tiles: 1024-byte atoms)
  uint8_t* store_bufs = smem + kStages * kPairStage;
  float* bias_bufs = reinterpret_cast<float*>(store_bufs + kPairEpi * 2 * kStoreBuf);
  float* ring = bias_bufs + kPairEpi * 128;
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(ring + 2 * kRing);  // (behind the first factors of wide scales)
  uint64_t* empty_bar = full_bar + kStages;
  uint64_t* accf_bar = empty_bar + kStages;
  uint64_t* acce_bar = accf_bar + 4;  // [k block & 1][half], as accf_bar
  uint64_t* sf_bar = acce_bar + 4;
  uint64_t* se_bar = sf_bar + 2;
  uint32_t* wide = reinterpret_cast<uint32_t*>(se_bar + 2);  // [group & 1][warp 2 or 3]: some of its scales may be wide
  uint32_t* tmem_slot = wide + 4;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // (uniform to the compiler)
  const int lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int tile0 = blockIdx.x >> 1, tile_step = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(&accf_bar[b], 1);
      mbar_init(&acce_bar[b], kPairEpi);  // half of the adding warps of each CTA
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sf_bar[b], 64);
      mbar_init(&se_bar[b], kPairEpi);
    }
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    if (p.vec) tma_prefetch_desc(&tmD);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  cluster_sync();  // the peer's barriers and tensor memory exist before anything targets them

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsHelp));
    if (warp == 0 && lane == 0) {
      int kc = 0, s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = tile0; tile < p.n_tiles && ok; tile += tile_step) {
        const int mt = tile / p.n_ntiles, nt = tile - mt * p.n_ntiles;
        for (int kb = 0; kb < p.num_kb; ++kb, ++kc) {
          if (kc >= kStages && !mbar_wait(&empty_bar[s], ph ^ 1u, p.fault, p.limit_ns, 71)) {
            ok = false;
            break;
          }
          uint8_t* a = smem + s * kPairStage;
          // both CTAs' tiles complete on the leader's barrier (the leader alone runs the MMAs)
          const uint32_t fb = cluster_map(smem_u32(&full_bar[s]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&full_bar[s], 2 * kPairStage);
          tma_load_2d_pair(a, &tmA, fb, kb * kKB, (2 * mt + rank) * kBlockM);
#pragma unroll
          for (int h = 0; h < 2; ++h)  // this CTA's 64 rows of each half
            tma_load_2d_pair(a + kTileBytes + h * (kTileBytes / 2), &tmB, fb, kb * kKB, nt * kPairBN + h * kHalf + rank * (kHalf / 2));
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // every load has landed and every commit has arrived before the CTA may exit
      if (rank == 0)
        for (int k = max(0, kc - kStages); k < kc; ++k)
          mbar_wait(&full_bar[k % kStages], (k / kStages) & 1, p.fault, p.limit_ns, 72);
      for (int k = max(0, kc - kStages); k < kc; ++k)
        mbar_wait(&empty_bar[k % kStages], (k / kStages) & 1, p.fault, p.limit_ns, 73);
    } else if (warp >= 2) {
      const int r = threadIdx.x - 64;  // rows r and r + 64
      // scales of a k block: A's of this thread's two rows, B's of the two halves; 1 where there is nothing (zeros, in range)
      const auto load_scales = [&](int tile, int kb, float* a, float* b) {
        const int mt = tile / p.n_ntiles, nt = tile - mt * p.n_ntiles;
        const int row = (2 * mt + rank) * kBlockM + r;
        const float* sa = p.sa + static_cast<int64_t>(kb) * p.M + row;
        const float* sb = p.sb + static_cast<int64_t>(kb) * p.nb + 2 * nt;
        a[0] = a[1] = b[1] = 1.f;
        if (row < p.M) a[0] = __ldg(sa);
        if (row + 64 < p.M) a[1] = __ldg(sa + 64);
        b[0] = __ldg(sb);
        if (2 * nt + 1 < p.nb) b[1] = __ldg(sb + 1);
      };
      const auto next_kb = [&](int& tile, int& kb) {
        if (++kb == p.num_kb) {
          kb = 0;
          tile += tile_step;
        }
      };
      int tile = tile0, kb = 0;
      for (int g = 0; tile < p.n_tiles; ++g) {
        int tile_g = tile, kb_g = kb;
        float va[kGroup][2], vb[kGroup][2];
#pragma unroll
        for (int i = 0; i < kGroup; ++i) {
          va[i][0] = va[i][1] = vb[i][0] = vb[i][1] = 1.f;
          if (tile < p.n_tiles) {
            load_scales(tile, kb, va[i], vb[i]);
            next_kb(tile, kb);
          }
        }
        // (one answer for the warp, which votes below)
        if (!__all_sync(0xffffffffu, g < 2 || mbar_wait(&se_bar[g & 1], ((g >> 1) - 1) & 1, p.fault, p.limit_ns, 77))) break;
        float* dst = ring + (g & 1) * (kGroup * 256) + r;
        // the ends of the magnitudes of each k block's products
        const auto ends = [&](auto of, float& lo, float& hi) {
          float l[kGroup], h[kGroup];
#pragma unroll
          for (int i = 0; i < kGroup; ++i) {
            const float a0 = fabsf(of(va[i][0])), a1 = fabsf(of(va[i][1])), b0 = fabsf(of(vb[i][0])), b1 = fabsf(of(vb[i][1]));
            l[i] = fminf(a0, a1) * fminf(b0, b1);
            h[i] = fmaxf(a0, a1) * fmaxf(b0, b1);
          }
          lo = fminf(fminf(l[0], l[1]), fminf(l[2], l[3]));
          hi = fmaxf(fmaxf(h[0], h[1]), fmaxf(h[2], h[3]));
        };
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) dst[i * 256 + j * 64] = va[i][j & 1] * vb[i][j >> 1];
        float lo, hi;
        ends([](float v) { return v; }, lo, hi);
        bool any = __any_sync(0xffffffffu, (lo < kMinNormal) | (hi > kMaxFinite));
        if (__builtin_expect(any, 0)) {  // the least scale multiplies as it is
          ends([](float v) { return one_for_least(v); }, lo, hi);
          any = __any_sync(0xffffffffu, (lo < kMinNormal) | (hi > kMaxFinite));
        }
        if (__builtin_expect(any, 0)) {  // wide scales (or zeros, infinities): read again, as kept in registers they spill
#pragma unroll 1
          for (int i = 0; i < kGroup && tile_g < p.n_tiles; ++i) {
            float a[2], b[2];
            load_scales(tile_g, kb_g, a, b);
            next_kb(tile_g, kb_g);
#pragma unroll
            for (int j = 0; j < 4; ++j) scale_factors(a[j & 1], b[j >> 1], dst[kRing + i * 256 + j * 64], dst[i * 256 + j * 64]);
          }
        }
        if (lane == 0) wide[(g & 1) * 2 + warp - 2] = any;
        mbar_arrive(&sf_bar[g & 1]);
      }
    } else if (warp == 1 && rank == 0 && elect_one()) {
      // (the columns behind K arrive as zeros: every k block is four MMAs)
      constexpr uint32_t idesc = idesc_e4m3_f32(2 * kBlockM, kHalf);
      const uint64_t desc0 = sdesc_kmajor_sw128(smem_u32(smem));
      const uint32_t desc_hi = static_cast<uint32_t>(desc0 >> 32);
      const uint32_t full0 = smem_u32(full_bar), empty0 = smem_u32(empty_bar), accf0 = smem_u32(accf_bar), acce0 = smem_u32(acce_bar);
      uint32_t lo = static_cast<uint32_t>(desc0), bar = 0, ph = 0;  // the stage: its tiles, its barriers' offset
      int it = 0;
      bool ok = true;
      for (int tile = tile0; tile < p.n_tiles && ok; tile += tile_step) {
        for (int kb = 0; kb < p.num_kb; ++kb, ++it) {
          const uint32_t b = it & 1, released = ((it >> 1) - 1) & 1;
          const bool ready = it >= 2 && mbar_try_three(full0 + bar, ph, acce0 + 16u * b, acce0 + 16u * b + 8u, released);
          if (!ready) ok = mbar_wait(&full_bar[bar >> 3], ph, p.fault, p.limit_ns, 75);
          const uint32_t d = tmem_base + 256u * b;
#pragma unroll
          for (uint32_t h = 0; h < 2; ++h) {
            if (!ready) {
              if (it >= 2) ok = ok && mbar_wait(&acce_bar[2 * b + h], released, p.fault, p.limit_ns, 74);
              if (!ok) break;
            }
            tc_fence_after();
            mma_kblock_pair(d + h * kHalf, lo, lo + (kTileBytes >> 4) + (kTileBytes / 2 >> 4) * h, desc_hi, idesc);
            commit_pair(accf0 + 16u * b + 8u * h);
          }
          if (!ok) break;
          commit_pair(empty0 + bar);
          bar += 8;
          lo += kPairStage >> 4;
          if (bar == 8 * kStages) {
            bar = 0;
            lo = static_cast<uint32_t>(desc0);
            ph ^= 1u;
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsAdd));
    const int q = warp & 3, half = (warp - 4) >> 2;  // TMEM lane quadrant this warp may access, half of the columns
    const uint32_t t0 = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(half * kHalf);
    const uint32_t scale0 = smem_u32(ring + half * 128 + q * 32 + lane);
    const uint32_t acce = cluster_map(smem_u32(&acce_bar[half]), 0), accf = smem_u32(&accf_bar[half]), sf0 = smem_u32(sf_bar);
    const uint32_t wide0 = smem_u32(wide + (q & 1));  // (rows q * 32 .. are warp 2 + (q & 1)'s)
    uint32_t plain = 0;  // the group's scales are there, and none of this warp's is wide
    int it = 0;
    for (int tile = tile0; tile < p.n_tiles; tile += tile_step) {
      F2 acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0;
      uint32_t u[32], v[32];
      {  // the bias of the warp's columns, on its way while the k blocks are added up
        const int n = (tile % p.n_ntiles) * kPairBN + half * kHalf + lane * 4;
        const uint32_t to = smem_u32(bias_bufs + (warp - 4) * kHalf + lane * 4);
        __syncwarp();  // the previous tile's has been read
#pragma unroll
        for (int i = 0; i < 4; ++i) copy4_async(to + 4u * i, p.bias ? p.bias + n + i : nullptr, p.bias && n + i < p.N);
      }
      const int end = it + p.num_kb;
      bool here = false;  // this k block's first loads are on their way
      for (; it < end; ++it) {
        const uint32_t b = it & 1;
        const uint32_t t = t0 + b * kPairBN;
        if (!here) {
          // (one answer for the warp, which the .aligned loads below want whole, also where some lanes' waits ran out)
          const bool ok = mbar_wait(&accf_bar[2 * b + half], (it >> 1) & 1, p.fault, p.limit_ns, 76);
          tc_fence_after();
          if (!__all_sync(0xffffffffu, ok && plain)) {
            if (!__all_sync(0xffffffffu, ok && mbar_wait(&sf_bar[(it / kGroup) & 1], (it / (2 * kGroup)) & 1, p.fault, p.limit_ns, 78)))
              break;
            plain = lds_u32(wide0 + 8u * ((it / kGroup) & 1)) == 0u;
            if (__builtin_expect(!__all_sync(0xffffffffu, plain), 0)) {
              const float f = lds_f32(scale0 + (it & (2 * kGroup - 1)) * 1024u + kRing * 4u);
              tmem_scale<kHalf>(t, [f](int) { return f; });
            }
          }
          tmem_ld_32x32b_x32(t, u);
          tmem_ld_32x32b_x32(t + 32u, v);
        }
        const float s = lds_f32(scale0 + (it & (2 * kGroup - 1)) * 1024u);
        const F2 s2 = f2(s, s);
        tmem_wait_x32(u);
        tmem_wait_x32(v);
        add_scaled(acc, u, s2);
        tmem_ld_32x32b_x32(t + 64u, u);
        add_scaled(acc + 16, v, s2);
        tmem_ld_32x32b_x32(t + 96u, v);
        tmem_wait_x32(u);
        tmem_wait_x32(v);
        tc_fence_before();
        __syncwarp();
        arrive_if(lane == 0, acce + 16u * b);
        const bool last = (it & (kGroup - 1)) == kGroup - 1;  // of the group
        if (last && lane == 0) mbar_arrive(&se_bar[(it / kGroup) & 1]);
        // the next k block, asked for now: where it is there, its loads leave between the last adds
        const int next = it + 1;
        const uint32_t turn = (next / kGroup) & 1;
        bool ready = mbar_test(accf + 16u * (b ^ 1), (next >> 1) & 1);
        if (last) plain = mbar_test(sf0 + 8u * turn, (next / (2 * kGroup)) & 1) && lds_u32(wide0 + 8u * turn) == 0u;
        ready = ready && plain && next < end;
        add_scaled(acc + 32, u, s2);
        here = __all_sync(0xffffffffu, ready);
        if (here) {
          tc_fence_after();
          tmem_ld_32x32b_x32(t0 + (b ^ 1) * kPairBN, u);
        }
        add_scaled(acc + 48, v, s2);
        if (here) tmem_ld_32x32b_x32(t0 + (b ^ 1) * kPairBN + 32u, v);
      }
      if (it < end) break;
      const int mt = tile / p.n_ntiles, nt = tile - mt * p.n_ntiles;
      const int row0 = (2 * mt + rank) * kBlockM + q * 32, n0 = nt * kPairBN + half * kHalf;
      uint8_t* buf = store_bufs + (warp - 4) * 2 * kStoreBuf;
      float* bias_s = bias_bufs + (warp - 4) * kHalf;
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      if (p.out_f32) store_sums<float>(p, &tmD, buf, bias_s, acc, row0, n0, lane);
      else store_sums<__nv_bfloat16>(p, &tmD, buf, bias_s, acc, row0, n0, lane);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (lane == 0) bulk_wait_read();  // the stores have left shared memory before the CTA exits
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();  // (one of its lanes comes from the issuing loop)
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
  cluster_sync();  // neither CTA leaves while the other may still write into it
}

// ================================================================================ few tiles or few rows: split K
// One CTA per (128 rows of B x kBN rows of A, part of K).  Up to 64 rows of A are the MMA's columns, B's rows its rows; with
// 128 it is the other way round, and a thread, which reads a row of the accumulator, has one scale per k block instead of one for
// each column, read from shared memory (512 x 4096 x 4096 17.9 us, this way 12.6).  Each CTA writes its sums
// into shared memory (over the stages, which are done with); the CTAs of a tile's cluster then each add up and store
// 1 / split of the tile's rows of D, reading the other CTAs' sums through distributed shared memory in a fixed order.
//
// What bounds it is latency, and for wide weights their bytes: the way to the first loads takes 1.1 us, the first data
// 1.2 more, the exchange about 1; the weights arrive in pieces of 128 bytes, a row each.  1 x 4096 x 4096 takes 7.2 us
// (its bytes 2.5), 64 x 8192 x 8192 18.0 (10.3), 512 x 4096 x 4096, 128 tiles of 128 x 128, 12.6 (4.6).  The tiles of 128 x
// 128 for few rows of A as well: 1 x 4096 x 4096 8.4, 32 x 8192 x 2048 8.9 for 7.9, 64 x 8192 x 8192 17.1, but 64 x 40000 x 1024
// 20.3 for 18.0 and 48 x 8192 x 2048 8.9 for 8.5.
namespace {
constexpr uint32_t kSumPitch = 132;  // floats per row of D of partial sums
template <int kBN> struct Split {
  static constexpr bool kRows = kBN == 128;                  // A's rows are the MMA's rows, B's its columns
  static constexpr int kEpi = kBN == 128 ? 8 : 4;            // warps that add up: one or two per lane quadrant
  static constexpr int kThreads = 32 * (2 + kEpi);
  static constexpr int kCols = kBN == 128 ? 64 : kBN;        // columns of the accumulator per warp
  static constexpr int kAcc = 4;                             // accumulators
  static constexpr uint32_t kStage = kTileBytes + kBN * kKB;
  static constexpr int kCtas = kBN == 128 ? 1 : 2;           // CTAs per SM
  static constexpr int kStages = kBN == 64 ? 4 : 5;
  // k blocks a step of the adding loop: with two, the scales stay in their registers from their loads to their use and no move
  // waits for the latest (32 x 4096 x 4096 7.9 us, this way 7.7, 24 x 8192 x 8192 16.4, 15.5; 64 columns spill: 48 x 8192 x
  // 2048 8.5, 9.0)
  static constexpr int kStep = kBN == 32 || kBN == 128 ? 2 : 1;
  static constexpr int kColScales = kRows ? 0 : kEpi * 2 * kCols;  // floats: [warp][k block & 1][column]
  static constexpr uint32_t kSmem = 1024u + kStages * kStage + kColScales * 4u + (2u * kStages + 2u * kAcc) * 8u + 16u;
  static_assert(kStages * kStage >= kBN * kSumPitch * 4u, "the sums lie over the stages");
  static_assert(kCtas * (kSmem + 1024u) <= 228u * 1024u, "shared memory");
};

// This CTA's rows of D, part, part + S, ...: the S CTAs' sums added up in order, scaled, stored; 4 columns per thread and
// item, 16 loads in flight.
template <int kThreads, int S>
VAE_DEV void add_parts_fp8(const Fp8GemmParams& p, uint32_t sums, int part, int m0, int rows, int n0) {
  constexpr int kItems = 16 / S;
  const int items = (rows - part + S - 1) / S * 32;  // (this CTA's rows) x 32 groups of columns
  const int lane = threadIdx.x & 31;
  const int n = n0 + lane * 4;
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
      const int64_t off = static_cast<int64_t>(m0 + r) * p.ldd + n;
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

template <int kBN>
__global__ void __launch_bounds__(Split<kBN>::kThreads, Split<kBN>::kCtas)
    gemm_fp8_split_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                          const __grid_constant__ Fp8GemmParams p) {
  using C = Split<kBN>;
  constexpr int kStages = C::kStages, kCols = C::kCols;
  constexpr int kAcc = C::kAcc;
  constexpr uint32_t kTmem = kAcc * kBN;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* col_bufs = reinterpret_cast<float*>(smem + kStages * C::kStage);
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(col_bufs + C::kColScales);
  uint64_t* empty_bar = full_bar + kStages;
  uint64_t* accf_bar = empty_bar + kStages;
  uint64_t* acce_bar = accf_bar + kAcc;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acce_bar + kAcc);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // (uniform to the compiler)
  const int lane = threadIdx.x & 31;
  const int tile = blockIdx.x / p.split, part = blockIdx.x - tile * p.split;
  const int mt = tile / p.n_ntiles, nt = tile - mt * p.n_ntiles;
  const int m0 = mt * kBN, n0 = nt * kBlockM;
  const int kb0 = static_cast<int>(static_cast<int64_t>(part) * p.num_kb / p.split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(part + 1) * p.num_kb / p.split);  // at least one k block

  const auto load_stage = [&](int s, int kb) {
    uint8_t* a = smem + s * C::kStage;
    mbar_arrive_expect_tx(&full_bar[s], C::kStage);
    tma_load_2d(a, &tmB, &full_bar[s], kb * kKB, n0);
    tma_load_2d(a + kTileBytes, &tmA, &full_bar[s], kb * kKB, m0);
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < kAcc; ++b) {
      mbar_init(&accf_bar[b], 1);
      mbar_init(&acce_bar[b], C::kEpi);
    }
    fence_barrier_init();
    // the first loads leave before the block meets (1 x 4096 x 4096: 7.3 us with them behind it)
    for (int s = 0; s < kStages && kb0 + s < kb1; ++s) load_stage(s, kb0 + s);
  }
  if (warp == 1) tmem_alloc(tmem_slot, kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  F2 acc[kCols / 2];
#pragma unroll
  for (int i = 0; i < kCols / 2; ++i) acc[i] = 0;
  const int q = warp & 3, half = (warp - 2) >> 2;  // (adding warps)
  if (warp == 0) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      int kb = min(kb0 + kStages, kb1);  // (the first ones are on their way)
      for (; kb < kb1; ++kb) {
        if (!mbar_wait(&empty_bar[s], ph, p.fault, p.limit_ns, 81)) break;
        load_stage(s, kb);
        if (++s == kStages) {
          s = 0;
          ph ^= 1u;
        }
      }
      const int n = kb - kb0;  // every load has landed before its memory is used for the sums
      for (int k = max(0, n - kStages); k < n; ++k)
        mbar_wait(&full_bar[k % kStages], (k / kStages) & 1, p.fault, p.limit_ns, 82);
    }
  } else if (warp == 1) {
    const uint32_t smem_base = smem_u32(smem);
    if (elect_one()) {
      constexpr uint32_t idesc = idesc_e4m3_f32(kBlockM, kBN);
      int s = 0, it = 0;
      uint32_t ph = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int b = it % kAcc;
        if ((it >= kAcc && !mbar_wait(&acce_bar[b], (it / kAcc - 1) & 1, p.fault, p.limit_ns, 83)) ||
            !mbar_wait(&full_bar[s], ph, p.fault, p.limit_ns, 84))
          break;
        tc_fence_after();
        const uint32_t a_addr = smem_base + static_cast<uint32_t>(s) * C::kStage;
        const uint64_t b_rows = sdesc_kmajor_sw128(a_addr), a_rows = sdesc_kmajor_sw128(a_addr + kTileBytes);
        const uint64_t adesc = C::kRows ? a_rows : b_rows, bdesc = C::kRows ? b_rows : a_rows;
#pragma unroll
        for (int k = 0; k < 4; ++k)  // (the columns behind K arrive as zeros)
          tc_mma_e4m3(tmem_base + static_cast<uint32_t>(b * kBN), adesc + 2u * k, bdesc + 2u * k, idesc, k > 0);
        tc_commit(&accf_bar[b]);
        tc_commit(&empty_bar[s]);
        if (++s == kStages) {
          s = 0;
          ph ^= 1u;
        }
      }
      // the MMAs are done before the CTA goes on (or given up on)
      if (it > 0) mbar_wait(&accf_bar[(it - 1) % kAcc], ((it - 1) / kAcc) & 1, p.fault, p.limit_ns, 85);
    }
    __syncwarp();
  } else {
    float* col_s = col_bufs + (warp - 2) * 2 * kCols;
    const uint32_t t0 = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(half * kCols);
    // scales of the next two k blocks: B's one, and A's for this lane's row, or its columns, lane and lane + 32
    constexpr int kL = !C::kRows && kCols > 32 ? 2 : 1;
    const int m = m0 + (C::kRows ? q * 32 : half * kCols) + lane;
    float qa[2][kL], qb[2];
    const auto fetch = [&](int kb, float* a, float& b) {
#pragma unroll
      for (int j = 0; j < kL; ++j) {
        a[j] = 1.f;  // (rows beyond A: zeros, whose scale is in range)
        if (kb < kb1 && lane + 32 * j < kCols && m + 32 * j < p.M) a[j] = __ldg(p.sa + static_cast<int64_t>(kb) * p.M + m + 32 * j);
      }
      b = kb < kb1 ? __ldg(p.sb + static_cast<int64_t>(kb) * p.nb + nt) : 1.f;
    };
    fetch(kb0, qa[0], qb[0]);
    fetch(kb0 + 1, qa[1], qb[1]);
    const uint32_t accf0 = smem_u32(accf_bar);
    bool ready = false;
    // adds up k block kb, whose scales are in slot h; those of kb + 2 then take their place (or, a k block a step, the last).
    // Not, if a wait ran out or a scale may be wide.
    const auto add = [&](int kb, int h) {
      const int it = kb - kb0, b = it % kAcc;
      float* cs = col_s + (it & 1) * kCols;
      F2 row_s = 0;
      bool plain = true;
#pragma unroll
      for (int j = 0; j < kL; ++j) {
        const float s = qa[h][j] * qb[h];
        plain &= in_range(one_for_least(qa[h][j]) * one_for_least(qb[h]));
        if constexpr (C::kRows) row_s = f2(s, s);
        else if (lane + 32 * j < kCols) cs[lane + 32 * j] = s;
      }
      if constexpr (!C::kRows) __syncwarp();
      if constexpr (C::kStep == 1) {
#pragma unroll
        for (int j = 0; j < kL; ++j) qa[0][j] = qa[1][j];
        qb[0] = qb[1];
        h = 1;
      }
      fetch(kb + 2, qa[h], qb[h]);
      const uint32_t t = t0 + static_cast<uint32_t>(b * kBN);
      if (!__all_sync(0xffffffffu, (ready || mbar_wait(&accf_bar[b], (it / kAcc) & 1, p.fault, p.limit_ns, 86)) && plain)) {
        if constexpr (C::kStep == 2) {
          return false;
        } else {
          if (!__all_sync(0xffffffffu, mbar_test(accf0 + 8u * b, (it / kAcc) & 1))) return false;
          tc_fence_after();
          float a[kL], bs;
          fetch(kb, a, bs);  // (again: kept until here they would take registers)
          const float2 s = tmem_scale_columns<kCols>(t, a[0], a[kL - 1], bs);
          if (lane < kCols) cs[lane] = s.x;
          if (kL == 2) cs[lane + 32] = s.y;
          __syncwarp();
        }
      }
      tc_fence_after();
      uint32_t raw[kCols];
      if constexpr (kCols == 16) {
        tmem_ld_32x32b_x16(t, raw);
        tmem_wait_x16(raw);
      } else {
#pragma unroll
        for (int j = 0; j < kCols; j += 32) tmem_ld_32x32b_x32(t + static_cast<uint32_t>(j), raw + j);
#pragma unroll
        for (int j = 0; j < kCols; j += 32) tmem_wait_x32(raw + j);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acce_bar[b]);
      ready = mbar_test(accf0 + 8u * ((it + 1) % kAcc), ((it + 1) / kAcc) & 1);  // answered when the adds are done
#pragma unroll
      for (int i = 0; i < kCols; i += 4) {
        F2 lo = row_s, hi = row_s;
        if constexpr (!C::kRows) {
          const float4 c = *reinterpret_cast<const float4*>(cs + i);
          lo = f2(c.x, c.y);
          hi = f2(c.z, c.w);
        }
        acc[i / 2] = f2_fma(f2_bits(raw[i], raw[i + 1]), lo, acc[i / 2]);
        acc[i / 2 + 1] = f2_fma(f2_bits(raw[i + 2], raw[i + 3]), hi, acc[i / 2 + 1]);
      }
      return true;
    };
    // The same for scales of any kind, a k block at a time: each sum times the first factor of its scales, then the second.
    // (From the first wide scale on, in place of add() where that takes two k blocks a step: in add(), as for one, 512 x
    // 4096 x 4096 takes 13.2 us for 12.4; for one a step this way 64 x 8192 x 8192 18.7 for 18.0.)
    const auto add_any = [&](int kb) {
      const int it = kb - kb0, b = it % kAcc;
      float first = 1.f, second = 1.f;
      {
        float a[kL], bs;
        fetch(kb, a, bs);
#pragma unroll
        for (int j = 0; j < kL; ++j) {
          scale_factors(a[j], bs, first, second);
          if (!C::kRows && lane + 32 * j < kCols) {
            col_s[lane + 32 * j] = first;
            col_s[kCols + lane + 32 * j] = second;
          }
        }
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&accf_bar[b], (it / kAcc) & 1, p.fault, p.limit_ns, 87))) return false;
      __syncwarp();
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < kCols; c += 16) {
        uint32_t raw[16];
        tmem_ld_32x32b_x16(t0 + static_cast<uint32_t>(b * kBN + c), raw);
        tmem_wait_x16(raw);
#pragma unroll
        for (int i = c; i < c + 16; i += 2) {
          const float2 f = C::kRows ? make_float2(first, first) : *reinterpret_cast<const float2*>(col_s + i);
          const float2 s = C::kRows ? make_float2(second, second) : *reinterpret_cast<const float2*>(col_s + kCols + i);
          acc[i / 2] = f2_fma(f2_mul(f2_bits(raw[i - c], raw[i - c + 1]), f2(f.x, f.y)), f2(s.x, s.y), acc[i / 2]);
        }
      }
      tc_fence_before();
      __syncwarp();  // (col_s has been read, too)
      if (lane == 0) mbar_arrive(&acce_bar[b]);
      return true;
    };
    int kb = kb0;
    for (; kb < kb1; kb += C::kStep) {
      if (!add(kb, 0)) break;
      if constexpr (C::kStep == 2) {
        if (kb + 1 >= kb1) continue;
        if (!add(kb + 1, 1)) {
          ++kb;
          break;
        }
      }
    }
    if constexpr (C::kStep == 2)
      for (; kb < kb1; ++kb)
        if (!add_any(kb)) break;
  }
  tc_fence_before();
  __syncthreads();  // loads landed, MMAs done (or given up on): the stages become the sums
  tc_fence_after();
  float* sums = reinterpret_cast<float*>(smem);
  if (warp >= 2) {
    if constexpr (C::kRows) {
      float* dst = sums + static_cast<uint32_t>(q * 32 + lane) * kSumPitch + half * kCols;
#pragma unroll
      for (int i = 0; i < kCols / 2; i += 2) {
        const float2 u = f2_get(acc[i]), v = f2_get(acc[i + 1]);
        *reinterpret_cast<float4*>(dst + 2 * i) = make_float4(u.x, u.y, v.x, v.y);
      }
    } else {
      float* dst = sums + static_cast<uint32_t>(half * kCols) * kSumPitch + q * 32 + lane;
#pragma unroll
      for (int i = 0; i < kCols / 2; ++i) {
        const float2 v = f2_get(acc[i]);
        dst[(2 * i) * kSumPitch] = v.x;
        dst[(2 * i + 1) * kSumPitch] = v.y;
      }
    }
  } else if (warp == 1) {
    tmem_dealloc(tmem_base, kTmem);
  }
  if (p.split > 1) cluster_sync();
  else __syncthreads();
  const int rows = min(kBN, p.M - m0);
  switch (p.split) {
    case 8: add_parts_fp8<C::kThreads, 8>(p, smem_u32(sums), part, m0, rows, n0); break;
    case 4: add_parts_fp8<C::kThreads, 4>(p, smem_u32(sums), part, m0, rows, n0); break;
    case 2: add_parts_fp8<C::kThreads, 2>(p, smem_u32(sums), part, m0, rows, n0); break;
    default: add_parts_fp8<C::kThreads, 1>(p, smem_u32(sums), part, m0, rows, n0); break;
  }
  if (p.split > 1) cluster_sync();  // no CTA leaves while another may still read its sums
}

// ================================================================================ host side
namespace {
using SplitKernel = void (*)(CUtensorMap, CUtensorMap, Fp8GemmParams);
struct SplitForm {
  int bn;
  SplitKernel kernel;
  int threads;
  uint32_t smem;
};
const SplitForm kSplitForms[4] = {
    {16, gemm_fp8_split_kernel<16>, Split<16>::kThreads, Split<16>::kSmem},
    {32, gemm_fp8_split_kernel<32>, Split<32>::kThreads, Split<32>::kSmem},
    {64, gemm_fp8_split_kernel<64>, Split<64>::kThreads, Split<64>::kSmem},
    {128, gemm_fp8_split_kernel<128>, Split<128>::kThreads, Split<128>::kSmem},
};

std::mutex g_mu;
struct DevInfo {
  bool ready = false;
  int n_sm = 0;
  int pairs = 0;        // pairs resident at once
  int clusters[4][4];   // by split form: clusters of 1, 2, 4, 8 CTAs resident at once
};
DevInfo g_dev[64];

cudaLaunchConfig_t cluster_config(cudaLaunchAttribute* attr, unsigned grid, unsigned cluster, int threads, size_t smem,
                                  cudaStream_t stream) {
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = cluster;
  attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
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
    e = cudaFuncSetAttribute(gemm_fp8_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    cudaLaunchConfig_t cfg = cluster_config(&attr, 2 * (d.n_sm / 2), 2, kPairThreads, kPairSmem, nullptr);
    // (a failed occupancy query is answered here, and its error with it)
    e = cudaOccupancyMaxActiveClusters(&d.pairs, gemm_fp8_pair_kernel, &cfg);
    if (e != cudaSuccess) cudaGetLastError();
    if (e != cudaSuccess || d.pairs <= 0) d.pairs = d.n_sm / 2;
    for (int f = 0; f < 4; ++f) {
      const SplitForm& sf = kSplitForms[f];
      e = cudaFuncSetAttribute(sf.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sf.smem));
      if (e != cudaSuccess) return e;
      for (int k = 0; k < 4; ++k) {
        cfg = cluster_config(&attr, 1u << k, 1u << k, sf.threads, sf.smem, nullptr);
        int mc = 0;
        if (cudaOccupancyMaxActiveClusters(&mc, sf.kernel, &cfg) != cudaSuccess) {
          cudaGetLastError();
          mc = 0;
        }
        d.clusters[f][k] = mc;
      }
    }
    d.ready = true;
  }
  *out = d;
  return cudaSuccess;
}

bool code_map(CUtensorMap* m, const void* base, int rows, int K, int box_rows) {
  // (the map ends at K: what lies in the codes' padding is not read)
  const uint64_t dims[2] = {static_cast<uint64_t>(K), static_cast<uint64_t>(rows)};
  const uint64_t strides[1] = {static_cast<uint64_t>(K + 15) / 16 * 16};
  const uint32_t box[2] = {kKB, static_cast<uint32_t>(box_rows)};
  return make_map(m, base, 2, dims, strides, box, 1);
}
}  // namespace

cudaError_t launch_gemm_fp8(const Fp8GemmArgs& a, cudaStream_t stream) {
  DevInfo dev;
  cudaError_t e = device_info(&dev);
  if (e != cudaSuccess) return e;
  Fp8GemmParams p{};
  p.M = a.M; p.N = a.N; p.K = a.K;
  p.num_kb = (a.K + kKB - 1) / kKB;
  p.nb = (a.N + kBlockM - 1) / kBlockM;
  p.alpha = a.alpha; p.sa = a.a_scales; p.sb = a.b_scales; p.bias = a.bias; p.y = a.y; p.out_f32 = a.out_f32; p.ldd = a.ldd;
  p.vec = (reinterpret_cast<uintptr_t>(a.y) & 15) == 0 && (a.ldd * (a.out_f32 ? 4 : 2)) % 16 == 0;
  p.whole16 = (static_cast<int64_t>(a.N) * (a.out_f32 ? 4 : 2)) % 16 == 0;
  p.fault = fault_word();
  p.limit_ns = wait_limit_ns();

  CUtensorMap tmA, tmB, tmD;
  cudaLaunchAttribute attr;
  // Up to 64 rows of A, or 128 x 128 tiles that fit the machine at once: the split kernel, K in as many parts (1, 2, 4 or
  // 8, a k block or more each) as still all run at once, or twice as many CTAs (the smaller forms fit an SM twice, but the
  // second ones start a microsecond later) where a part's weights still take longer than the exchange, which grows with
  // the rows of A: 1 x 4096 x 4096 in 8 parts for 4 6.8 us for 7.6, 64 x 8192 x 8192 in 4 for 2 18.2 for 19.1, but
  // 48 x 8192 x 2048 in 4 for 2 9.2 for 8.5 and 8 x 2048 x 2048 in 8 for 4 5.1 for 4.9.
  // One wave of 128 x 128 tiles against pairs: 512 x 4096 x 4096 12.6 us for 17.9, 2432 x 1024 x 256 5.9 for 6.5; two waves:
  // 3520 x 1024 x 1024 12.6 for 9.2, 640 x 4096 x 4096 23.1 for 18.4.
  const int form = a.M <= 16 ? 0 : a.M <= 32 ? 1 : a.M <= 64 ? 2 : 3;
  const int64_t mtiles = (static_cast<int64_t>(a.M) + kSplitForms[form].bn - 1) / kSplitForms[form].bn;
  const int64_t tiles128 = mtiles * p.nb;
  if (form < 3 || tiles128 <= dev.n_sm) {
    const SplitForm& sf = kSplitForms[form];
    int parts = 1;
    for (int k = 3; k >= 1 && parts == 1; --k) {
      const bool once = tiles128 <= dev.clusters[form][k];
      const bool twice = form < 3 && (tiles128 << k) <= dev.n_sm * 7 / 4 && (p.num_kb >> k) * 4 >= sf.bn;
      if ((once || twice) && (1 << k) <= p.num_kb) parts = 1 << k;
    }
    if (!code_map(&tmA, a.a_codes, a.M, a.K, sf.bn) || !code_map(&tmB, a.b_codes, a.N, a.K, kBlockM)) return cudaErrorInvalidValue;
    p.n_ntiles = p.nb;
    p.n_tiles = static_cast<int>(tiles128);
    p.split = parts;
    cudaLaunchConfig_t cfg = cluster_config(&attr, static_cast<unsigned>(p.n_tiles * p.split), static_cast<unsigned>(parts),
                                            sf.threads, sf.smem, stream);
    return cudaLaunchKernelEx(&cfg, sf.kernel, tmA, tmB, p);
  }
  memset(&tmD, 0, sizeof(tmD));
  if (!code_map(&tmA, a.a_codes, a.M, a.K, kBlockM) || !code_map(&tmB, a.b_codes, a.N, a.K, kHalf / 2))
    return cudaErrorInvalidValue;
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
  const unsigned pairs = static_cast<unsigned>(std::min<int64_t>(tiles, dev.pairs));
  cudaLaunchConfig_t cfg = cluster_config(&attr, 2 * pairs, 2, kPairThreads, kPairSmem, stream);
  return cudaLaunchKernelEx(&cfg, gemm_fp8_pair_kernel, tmA, tmB, tmD, p);
}

}  // namespace vae
