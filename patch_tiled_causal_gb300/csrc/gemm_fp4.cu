// Product of two microscaled 4-bit operands on the 5th-generation tensor cores (tcgen05, sm_103a):
//   D[m, n] = alpha * sum_k (a[m, k] sa[m, k / block]) (b[n, k] sb[n, k / block]) + bias[n]
// with e2m1 a, b and power-of-two (MXFP4, block 32) or e4m3 (NVFP4, block 16) scales, which the tensor cores
// apply to the products of each block before the fp32 accumulation (kind::mxf4, kind::mxf4nvf4).
//
// A k block is 256 columns: 128 bytes of codes per row, which one TMA box brings into a 128-byte-swizzled
// K-major tile, and 8 (MXFP4) or 16 (NVFP4) scale bytes per row, which arrive as whole 128-row x 4-block tiles
// of 512 bytes and go from shared into tensor memory with tcgen05.cp (32 lanes x 16 bytes, repeated for the
// four lane quadrants).  Each MMA takes 64 columns.  Rows and columns beyond the operands arrive as
// zeros, and the MMAs of the last k block stop at K, so any size works without padding.
#include <algorithm>
#include <cstring>
#include <mutex>

#include "common.cuh"
#include "fp4.cuh"
#include "internal.h"

namespace vae {

struct Fp4GemmParams {
  int M, N, K;
  int num_kb;         // k blocks of 256 columns
  int n_ntiles, n_tiles;
  float alpha;
  const float* bias;
  void* y;
  int out_f32;
  int vec;            // rows of D start on 16-byte boundaries
  int64_t ldd;
  uint32_t* fault;
  uint64_t limit_ns;
};

namespace {

constexpr int kThreads = 192;
constexpr int kBlockM = 128;
constexpr int kBN = 128;
constexpr int kKB = 256;                          // columns per k block
constexpr uint32_t kTileBytes = kBlockM * kKB / 2;  // codes of 128 rows
constexpr int kStages = 5;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSfCol = 256;                  // scale factors behind the two accumulators

template <int kFmt> constexpr int kGroups = kFmt == VAE_MXFP4 ? 2 : 4;  // 4-block scale groups per k block
template <int kFmt> constexpr uint32_t kStageBytes = 2u * kTileBytes + 2u * kGroups<kFmt> * 512u;

// D[tmem] (+)= A B^T with block scales in tensor memory, 64 columns of K.
template <int kFmt>
VAE_DEV void tc_mma_fp4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                        uint32_t accumulate) {
  if constexpr (kFmt == VAE_MXFP4) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  }
}

// One 512-byte scale tile from shared into 4 columns of tensor memory.
VAE_DEV void tc_cp_scales(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
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

// 32 columns of one row of D.
VAE_DEV void store_chunk(const Fp4GemmParams& p, int row, int n0, const uint32_t* raw) {
  if (row >= p.M || n0 >= p.N) return;
  float v[32];
#pragma unroll
  for (int i = 0; i < 32; ++i)
    v[i] = __uint_as_float(raw[i]) * p.alpha + (p.bias ? __ldg(p.bias + min(n0 + i, p.N - 1)) : 0.f);
  const int64_t off = static_cast<int64_t>(row) * p.ldd + n0;
  if (p.vec && n0 + 32 <= p.N) {
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
      if (p.out_f32) store8(static_cast<float*>(p.y) + off + i, v + i);
      else store8(static_cast<__nv_bfloat16*>(p.y) + off + i, v + i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (n0 + i >= p.N) break;
      if (p.out_f32) static_cast<float*>(p.y)[off + i] = v[i];
      else static_cast<__nv_bfloat16*>(p.y)[off + i] = f2bf(v[i]);
    }
  }
}

}  // namespace

// Persistent: each CTA walks 128 x 128 tiles (the N tiles of one M tile next to each other, so that A is read from L2).
// Warp 0 loads, warp 1 owns the tensor memory and issues, warps 2..5 drain the accumulators; two accumulators
// let the epilogue of a tile overlap the MMAs of the next.  The scales of stage s live in their own columns of
// tensor memory: the copy that overwrites them is issued after the barrier that says the stage's MMAs are done.
template <int kFmt>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_fp4_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                    const __grid_constant__ Fp4GemmParams p) {
  constexpr int kG = kGroups<kFmt>;
  constexpr uint32_t kStage = kStageBytes<kFmt>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + kStages * kStage);
  uint64_t* empty_bar = full_bar + kStages;
  uint64_t* accf_bar = empty_bar + kStages;
  uint64_t* acce_bar = accf_bar + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acce_bar + 2);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&accf_bar[a], 1);
      mbar_init(&acce_bar[a], 4 * 32);
    }
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSA);
    tma_prefetch_desc(&tmSB);
  }
  if (warp == 1) tmem_alloc(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      int kc = 0, s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < p.n_tiles && ok; tile += gridDim.x) {
        const int mt = tile / p.n_ntiles, nt = tile - mt * p.n_ntiles;
        for (int kb = 0; kb < p.num_kb; ++kb, ++kc) {
          if (kc >= kStages && !mbar_wait(&empty_bar[s], ph ^ 1u, p.fault, p.limit_ns, 51)) {
            ok = false;
            break;
          }
          uint8_t* a = smem + s * kStage;
          uint8_t* b = a + kTileBytes;
          uint8_t* sa = b + kTileBytes;
          uint8_t* sb = sa + kG * 512;
          mbar_arrive_expect_tx(&full_bar[s], kStage);
          tma_load_2d(a, &tmA, &full_bar[s], kb * (kKB / 2), mt * kBlockM);
          tma_load_2d(b, &tmB, &full_bar[s], kb * (kKB / 2), nt * kBN);
          tma_load_3d(sa, &tmSA, &full_bar[s], 0, kb * kG, mt);
          tma_load_3d(sb, &tmSB, &full_bar[s], 0, kb * kG, nt);
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      for (int k = max(0, kc - kStages); k < kc; ++k)  // every load has landed before the block may exit
        mbar_wait(&full_bar[k % kStages], (k / kStages) & 1, p.fault, p.limit_ns, 52);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t smem_base = smem_u32(smem);
      int s = 0, it = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < p.n_tiles && ok; tile += gridDim.x, ++it) {
        const int acc = it & 1, u = it >> 1;
        if (u > 0 && !mbar_wait(&acce_bar[acc], (u - 1) & 1, p.fault, p.limit_ns, 56)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kBN);
        for (int kb = 0; kb < p.num_kb; ++kb) {
          if (!mbar_wait(&full_bar[s], ph, p.fault, p.limit_ns, 53)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_addr = smem_base + static_cast<uint32_t>(s) * kStage;
          const uint32_t sa_addr = a_addr + 2u * kTileBytes;
          const uint32_t sfa = tmem_base + kSfCol + static_cast<uint32_t>(s) * (8u * kG);
          const uint32_t sfb = sfa + 4u * kG;
#pragma unroll
          for (uint32_t g = 0; g < kG; ++g) {
            tc_cp_scales(sfa + 4u * g, sdesc_scales(sa_addr + g * 512u));
            tc_cp_scales(sfb + 4u * g, sdesc_scales(sa_addr + (kG + g) * 512u));
          }
          const uint64_t adesc = sdesc_kmajor_sw128(a_addr);
          const uint64_t bdesc = sdesc_kmajor_sw128(a_addr + kTileBytes);
          const int steps = min(4, (p.K - kb * kKB + 63) / 64);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k >= steps) break;
            const uint32_t g = kFmt == VAE_MXFP4 ? k >> 1 : k;
            const uint32_t id = kFmt == VAE_MXFP4 ? (k & 1) * 2 : 0;
            tc_mma_fp4<kFmt>(d_tmem, adesc + 2u * k, bdesc + 2u * k, idesc_fp4<kFmt>(kBlockM, kBN, id), sfa + 4u * g,
                             sfb + 4u * g, (kb == 0 && k == 0) ? 0u : 1u);
          }
          tc_commit(&empty_bar[s]);
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
        tc_commit(&accf_bar[acc]);
      }
    }
  } else {
    const int q = warp & 3;  // TMEM lane quadrant this warp may access
    int it = 0;
    for (int tile = blockIdx.x; tile < p.n_tiles; tile += gridDim.x, ++it) {
      const int acc = it & 1, u = it >> 1;
      if (!mbar_wait(&accf_bar[acc], u & 1, p.fault, p.limit_ns, 55)) break;
      tc_fence_after();
      const int mt = tile / p.n_ntiles, nt = tile - mt * p.n_ntiles;
      const int row = mt * kBlockM + q * 32 + lane;
      for (int j = 0; j < kBN / 32; ++j) {
        uint32_t raw[32];
        tmem_ld_32x32b_x32(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * kBN + j * 32), raw);
        tmem_ld_wait();
        if (j == kBN / 32 - 1) {
          tc_fence_before();
          mbar_arrive(&acce_bar[acc]);
        }
        store_chunk(p, row, nt * kBN + j * 32, raw);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

// ================================================================================ host side
namespace {
std::mutex g_mu;
struct DevInfo {
  bool ready = false;
  int n_sm = 0;
};
DevInfo g_dev[64];
}  // namespace

cudaError_t launch_gemm_fp4(const Fp4GemmArgs& a, cudaStream_t stream) {
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    DevInfo& d = g_dev[dev];
    if (!d.ready) {
      e = cudaDeviceGetAttribute(&d.n_sm, cudaDevAttrMultiProcessorCount, dev);
      if (e != cudaSuccess) return e;
      for (auto* k : {gemm_fp4_kernel<VAE_MXFP4>, gemm_fp4_kernel<VAE_NVFP4>}) {
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        if (e != cudaSuccess) return e;
      }
      d.ready = true;
    }
    n_sm = d.n_sm;
  }
  const bool mx = a.format == VAE_MXFP4;
  Fp4GemmParams p{};
  p.M = a.M; p.N = a.N; p.K = a.K;
  p.num_kb = (a.K + kKB - 1) / kKB;
  p.n_ntiles = (a.N + kBN - 1) / kBN;
  const int64_t mtiles = (static_cast<int64_t>(a.M) + kBlockM - 1) / kBlockM;
  if (mtiles * p.n_ntiles > 0x40000000LL) return cudaErrorInvalidValue;
  p.n_tiles = static_cast<int>(mtiles * p.n_ntiles);
  p.alpha = a.alpha; p.bias = a.bias; p.y = a.y; p.out_f32 = a.out_f32; p.ldd = a.ldd;
  p.vec = (reinterpret_cast<uintptr_t>(a.y) & 15) == 0 && (a.ldd * (a.out_f32 ? 4 : 2)) % 16 == 0;
  p.fault = fault_word();
  p.limit_ns = wait_limit_ns();

  const uint64_t pitch = static_cast<uint64_t>(a.K + 31) / 32 * 16;
  const uint64_t groups = static_cast<uint64_t>(fp4_groups(a.format, a.K));
  const uint32_t kg = mx ? kGroups<VAE_MXFP4> : kGroups<VAE_NVFP4>;
  CUtensorMap tmA, tmB, tmSA, tmSB;
  auto code_map = [&](CUtensorMap* m, const void* base, int rows, uint32_t box_rows) {
    const uint64_t dims[2] = {pitch, static_cast<uint64_t>(rows)};
    const uint64_t strides[1] = {pitch};
    const uint32_t box[2] = {kKB / 2, box_rows};
    return make_map(m, base, 2, dims, strides, box, 1);
  };
  auto scale_map = [&](CUtensorMap* m, const void* base, int rows, uint32_t box_tiles) {
    const uint64_t dims[3] = {128, groups, (static_cast<uint64_t>(rows) + 127) / 128};
    const uint64_t strides[2] = {512, 512 * groups};
    const uint32_t box[3] = {128, kg, box_tiles};
    return make_map(m, base, 3, dims, strides, box, 4, false);
  };
  if (!code_map(&tmA, a.a_codes, a.M, kBlockM) || !code_map(&tmB, a.b_codes, a.N, kBN) ||
      !scale_map(&tmSA, a.a_scales, a.M, 1) || !scale_map(&tmSB, a.b_scales, a.N, 1))
    return cudaErrorInvalidValue;
  const uint32_t stage = mx ? kStageBytes<VAE_MXFP4> : kStageBytes<VAE_NVFP4>;
  const size_t smem = 1024 + static_cast<size_t>(kStages) * stage + (2 * kStages + 4) * 8 + 16;
  const unsigned grid = static_cast<unsigned>(std::min(p.n_tiles, n_sm));
  if (mx) gemm_fp4_kernel<VAE_MXFP4><<<grid, kThreads, smem, stream>>>(tmA, tmB, tmSA, tmSB, p);
  else gemm_fp4_kernel<VAE_NVFP4><<<grid, kThreads, smem, stream>>>(tmA, tmB, tmSA, tmSB, p);
  return cudaGetLastError();
}

}  // namespace vae
