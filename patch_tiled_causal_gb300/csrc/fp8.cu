// 8-bit operands with block scales: quantisation, reading back, the channel RMS norm of a residual sum that writes
// them, and the entry points.
//
// TensorRT-LLM PR #16066 "ParallelVAE_TrtllmWan for native Wan VAE" (reviewer comment) names low-precision quantisation
// with the norm fused into it; these operands lie between bf16 and the 4-bit ones: e4m3 with an fp32 scale for each
// block of 128.  The product is in gemm_fp8.cu.
#include <cstdarg>
#include <cstdio>

#include "fp8.cuh"
#include "internal.h"

namespace vae {
namespace {

constexpr int kThreads = 256;
constexpr int kVpt = 2;            // vectors of 16 values in flight per thread
constexpr int kMaxCols = 1 << 18;  // a vector index inside a block times vpr stays below 2^32 (vpr_magic)

struct Fp8Params {
  const void* x;         // quantise: values in; read back: codes in
  void* y;               // quantise: codes out; read back: values out
  float* scales;         // [column blocks][row_blocks]
  int64_t ld;            // elements between rows of the values
  int rows, cols;
  int pitch;             // bytes between rows of the codes
  int row_blocks;        // scales per column block
  int row_shift;         // row >> row_shift is a row's row block
  int vpr;               // vectors (of 16 columns) handled per row
  uint32_t vpr_magic;    // ceil(2^32 / vpr)
  uint64_t vpr_magic64;  // ceil(2^64 / vpr) (vpr >= 2)
  int a32;               // rows of the values start on 32-byte boundaries
  uint32_t* fault;
};

// First vector of this block -> (row, vector in its row); the block's later vectors then need 32 bits only.
VAE_DEV void block_origin(const Fp8Params& p, int& row0, uint32_t& rem0) {
  const int64_t base = static_cast<int64_t>(blockIdx.x) * (kThreads * kVpt);
  const int64_t r = p.vpr == 1 ? base : static_cast<int64_t>(__umul64hi(static_cast<uint64_t>(base), p.vpr_magic64));
  row0 = static_cast<int>(r);
  rem0 = static_cast<uint32_t>(base - r * p.vpr);
}

// The vector at (row, col) of a matrix of rows x cols values, zeros outside it.  kVec: rows start on 16-byte boundaries;
// otherwise the warp reads its elements 32 adjacent ones at a time and hands them out through shared memory (sh: 512
// elements of the warp's own).  The whole warp calls it.
template <typename T, bool kVec>
VAE_DEV void load_vec(LaneVec<T>& in, const T* x, int64_t ld, int rows, int cols, int row, int col, bool a32, T* sh) {
  if constexpr (kVec) {
    in.zero();
    if (row < rows && col < cols) {
      const T* src = x + row * ld + col;
      if (col + kLane <= cols) {
        in.load(src, a32);
      } else {
#pragma unroll
        for (int i = 0; i < kLane; ++i)
          if (col + i < cols) reinterpret_cast<T*>(in.w)[i] = src[i];
      }
    }
  } else {
    const int lane = threadIdx.x & 31;
    T e[kLane];
#pragma unroll
    for (int i = 0; i < kLane; ++i) {
      int er, ec;
      element_of(i, lane, row, col, er, ec);
      e[i] = from_f<T>(0.f);
      if (er < rows && ec < cols) e[i] = x[er * ld + ec];
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kLane; ++i) sh[i * 32 + lane] = e[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < LaneVec<T>::kW; i += 4) {
      const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(sh + lane * kLane) + i);
      in.w[i] = u.x; in.w[i + 1] = u.y; in.w[i + 2] = u.z; in.w[i + 3] = u.w;
    }
  }
}

// A lane's 16 values to (row, col) of a matrix, as T; as above.
template <typename T, bool kVec>
VAE_DEV void store_vec(T* y, const float* v, int64_t ld, int rows, int cols, int row, int col, bool a32, T* sh) {
  if constexpr (kVec) {
    if (row >= rows || col >= cols) return;
    T* dst = y + row * ld + col;
    if (col + kLane <= cols) {
      store_lane(dst, v, a32);
    } else {
#pragma unroll
      for (int i = 0; i < kLane; ++i)
        if (col + i < cols) dst[i] = from_f<T>(v[i]);
    }
  } else {
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kLane; i += 8) store8(sh + lane * kLane + i, v + i);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kLane; ++i) {
      int er, ec;
      element_of(i, lane, row, col, er, ec);
      if (er < rows && ec < cols) y[er * ld + ec] = sh[i * 32 + lane];
    }
  }
}

// The warp's staging area for rows that start anywhere (512 values; next to nothing where none is needed).
#define VAE_STAGE(T, kVec, threads)                                                                       \
  __shared__ __align__(16) uint8_t stage_[(kVec) ? 1 : (threads) / 32][(kVec) ? 16 : 512 * sizeof(T)]; \
  uint8_t* const stage = stage_[(kVec) ? 0 : threadIdx.x >> 5]

}  // namespace

// One scale per 128 columns of a row.  One vector of 16 columns per lane and step, 8 lanes per block; the vectors of a
// row run to the end of its last block.  HBM-bound by its bytes (x read once, 1 + 1/32 bytes per value written).
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) quantize_fp8_kernel(const __grid_constant__ Fp8Params p) {
  VAE_STAGE(T, kVec, kThreads);
  int row0;
  uint32_t rem0;
  block_origin(p, row0, rem0);
  int row[kVpt], col[kVpt];
  LaneVec<T> in[kVpt];
#pragma unroll
  for (int k = 0; k < kVpt; ++k) {
    const uint32_t idx = rem0 + static_cast<uint32_t>(k * kThreads) + threadIdx.x;
    const uint32_t r = __umulhi(idx, p.vpr_magic);  // (vpr >= 8 here)
    row[k] = row0 + static_cast<int>(r);
    col[k] = static_cast<int>(idx - r * static_cast<uint32_t>(p.vpr)) * kLane;
    load_vec<T, kVec>(in[k], static_cast<const T*>(p.x), p.ld, p.rows, p.cols, row[k], col[k], p.a32, reinterpret_cast<T*>(stage));
  }
  bool ok = true;
#pragma unroll
  for (int k = 0; k < kVpt; ++k) {
    F2 v[kLane / 2];
    in[k].get(v);
    const Fp8Scale q = fp8_scale(team_amax(lane_amax(v)));
    const uint4 codes = fp8_codes(v, q);
    ok = ok && q.finite;
    if (row[k] < p.rows) {
      if (col[k] < p.pitch)
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.y) + static_cast<int64_t>(row[k]) * p.pitch + col[k]) = codes;
      if ((threadIdx.x & (kFp8Team - 1)) == 0)
        p.scales[static_cast<int64_t>(col[k] / kFp8Block) * p.row_blocks + row[k]] = q.s;
    }
  }
  if (!ok) raise_fault(p.fault, FAULT_RANGE, 45);
}

// One scale per 128 columns of 128 rows: a thread block per block of values, which stays in registers (64 values a
// thread) between its maximum and its codes.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) quantize_fp8_block_kernel(const __grid_constant__ Fp8Params p) {
  VAE_STAGE(T, kVec, kThreads);
  constexpr int kV = kFp8Block * kFp8Team / kThreads;
  const int nc = p.vpr / kFp8Team;  // column blocks
  const int rb = blockIdx.x / nc, cb = blockIdx.x - rb * nc;
  const int row = rb * kFp8Block + threadIdx.x / kFp8Team, col = cb * kFp8Block + threadIdx.x % kFp8Team * kLane;
  constexpr int kStep = kThreads / kFp8Team;
  LaneVec<T> in[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i)
    load_vec<T, kVec>(in[i], static_cast<const T*>(p.x), p.ld, p.rows, p.cols, row + i * kStep, col, p.a32, reinterpret_cast<T*>(stage));
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    F2 v[kLane / 2];
    in[i].get(v);
    m = max_abs_or_nan(m, lane_amax(v), 0.f);
  }
#pragma unroll
  for (int d = 1; d < 32; d *= 2) m = max_abs_or_nan(m, __shfl_xor_sync(0xffffffffu, m, d), 0.f);
  __shared__ float part[kThreads / 32];
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) m = max_abs_or_nan(m, part[i], 0.f);
  const Fp8Scale q = fp8_scale(m);
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int r = row + i * kStep;
    if (r >= p.rows || col >= p.pitch) continue;
    F2 v[kLane / 2];
    in[i].get(v);
    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.y) + static_cast<int64_t>(r) * p.pitch + col) = fp8_codes(v, q);
  }
  if (threadIdx.x == 0) {
    p.scales[static_cast<int64_t>(cb) * p.row_blocks + rb] = q.s;
    if (!q.finite) raise_fault(p.fault, FAULT_RANGE, 46);
  }
}

// Values of codes: one vector of 16 columns per lane and step.  HBM-bound like the quantisation.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) dequantize_fp8_kernel(const __grid_constant__ Fp8Params p) {
  VAE_STAGE(T, kVec, kThreads);
  int row0;
  uint32_t rem0;
  block_origin(p, row0, rem0);
  int row[kVpt], col[kVpt];
  uint4 c[kVpt];
  float s[kVpt];
#pragma unroll
  for (int k = 0; k < kVpt; ++k) {
    const uint32_t idx = rem0 + static_cast<uint32_t>(k * kThreads) + threadIdx.x;
    const uint32_t q = p.vpr == 1 ? idx : __umulhi(idx, p.vpr_magic);
    col[k] = static_cast<int>(idx - q * static_cast<uint32_t>(p.vpr)) * kLane;
    row[k] = row0 + static_cast<int>(q);
    c[k] = make_uint4(0u, 0u, 0u, 0u);
    s[k] = 0.f;
    if (row[k] < p.rows) {
      c[k] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.x) +
                                                   static_cast<int64_t>(row[k]) * p.pitch + col[k]));
      s[k] = __ldg(p.scales + static_cast<int64_t>(col[k] / kFp8Block) * p.row_blocks + (row[k] >> p.row_shift));
    }
  }
#pragma unroll
  for (int k = 0; k < kVpt; ++k) {
    float v[kLane];
    e4m3x4_values(c[k].x, v);
    e4m3x4_values(c[k].y, v + 4);
    e4m3x4_values(c[k].z, v + 8);
    e4m3x4_values(c[k].w, v + 12);
#pragma unroll
    for (int i = 0; i < kLane; ++i) v[i] *= s[k];
    store_vec<T, kVec>(static_cast<T*>(p.y), v, p.ld, p.rows, p.cols, row[k], col[k], p.a32, reinterpret_cast<T*>(stage));
  }
}

// ================================================================================ RMS norm of a residual sum
namespace {
constexpr int kRmsMaxCols = 32768;  // 2048 vectors: two for each of 1024 threads (four for 512 through shared memory)

struct Fp8RmsParams {
  const void* x; const void* residual; void* total;  // residual, total: may be null
  const float* gamma; const float* beta;             // beta: may be null
  uint8_t* codes; float* scales;
  int64_t ld_x, ld_residual, ld_total;
  int rows, cols, pitch;
  float eps, inv_cols;
  int silu;
  int ax32, ar32, at32;  // rows of x, the residual, the total start on 32-byte boundaries
  int pvec;              // gamma and beta are 16-byte aligned
  uint32_t* fault;
};

// 16 parameters from col on, `fill` behind the last column
VAE_DEV void load_params(F2* v, const float* src, int col, int cols, bool vec) {
  if (vec && col + kLane <= cols) {
#pragma unroll
    for (int i = 0; i < kLane / 4; ++i) {
      const float4 t = __ldg(reinterpret_cast<const float4*>(src + col) + i);
      v[2 * i] = f2(t.x, t.y);
      v[2 * i + 1] = f2(t.z, t.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kLane / 2; ++i)
      v[i] = f2(col + 2 * i < cols ? __ldg(src + col + 2 * i) : 0.f,
                col + 2 * i + 1 < cols ? __ldg(src + col + 2 * i + 1) : 0.f);
  }
}
}  // namespace

// h = x + residual (fp32), total = h rounded, y = SiLU(h / sqrt(mean h^2 + eps) * gamma + beta), y quantised with one
// scale per 128 columns.  The norm takes h before its rounding: the total's own rounding touches the total only.
// kTeam threads hold a row between its two passes (sum of squares, normalisation), kVecs vectors of 16 columns each, so
// everything is read and written once: HBM-bound.  kTeam <= 32: rows share a warp; kTeam = 0: the whole thread block
// holds one row.  A row whose squares leave fp32 comes out as NaN, and raises VAE_ERR_RANGE with it.
template <typename TX, typename TR, bool kVec, int kTeam, int kVecs>
__global__ void __launch_bounds__(kTeam ? kThreads : kRmsMaxCols / kLane / kVecs)
    residual_rms_fp8_kernel(const __grid_constant__ Fp8RmsParams p) {
  VAE_STAGE(float, kVec, kTeam ? kThreads : kRmsMaxCols / kLane / kVecs);
  const int team = kTeam ? kTeam : static_cast<int>(blockDim.x);
  const int t = kTeam ? threadIdx.x % (kTeam ? kTeam : 1) : threadIdx.x;
  const int row = kTeam ? static_cast<int>(blockIdx.x) * (kThreads / (kTeam ? kTeam : 1)) + threadIdx.x / (kTeam ? kTeam : 1)
                        : static_cast<int>(blockIdx.x);
  F2 h[kVecs][kLane / 2];
  {
    LaneVec<TX> x[kVecs];
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
      load_vec<TX, kVec>(x[k], static_cast<const TX*>(p.x), p.ld_x, p.rows, p.cols, row, (k * team + t) * kLane, p.ax32, reinterpret_cast<TX*>(stage));
    if (p.residual) {
      LaneVec<TR> r[kVecs];
#pragma unroll
      for (int k = 0; k < kVecs; ++k)
        load_vec<TR, kVec>(r[k], static_cast<const TR*>(p.residual), p.ld_residual, p.rows, p.cols, row,
                           (k * team + t) * kLane, p.ar32, reinterpret_cast<TR*>(stage));
#pragma unroll
      for (int k = 0; k < kVecs; ++k) {
        F2 u[kLane / 2];
        x[k].get(h[k]);
        r[k].get(u);
#pragma unroll
        for (int i = 0; i < kLane / 2; ++i) h[k][i] = f2_add(h[k][i], u[i]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kVecs; ++k) x[k].get(h[k]);
    }
  }
  F2 s2 = f2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kVecs; ++k)
#pragma unroll
    for (int i = 0; i < kLane / 2; ++i) s2 = f2_fma(h[k][i], h[k][i], s2);
  float2 sp = f2_get(s2);
  float ss = sp.x + sp.y;
#pragma unroll
  for (int d = 1; d < (kTeam ? kTeam : 32); d *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, d);
  if constexpr (kTeam == 0) {
    __shared__ float part[32];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
    __syncthreads();
    ss = 0.f;
    for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) ss += part[i];
  }
  if (p.total) {
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      float v[kLane];
#pragma unroll
      for (int i = 0; i < kLane / 2; ++i) {
        const float2 u = f2_get(h[k][i]);
        v[2 * i] = u.x;
        v[2 * i + 1] = u.y;
      }
      store_vec<TR, kVec>(static_cast<TR*>(p.total), v, p.ld_total, p.rows, p.cols, row, (k * team + t) * kLane, p.at32,
                          reinterpret_cast<TR*>(stage));
    }
  }
  const float r = ss <= 3.402823466e38f ? __frcp_rn(__fsqrt_rn(fmaf(ss, p.inv_cols, p.eps))) : __int_as_float(0x7fffffff);
  bool ok = true;
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    const int col = (k * team + t) * kLane;
    F2 g[kLane / 2];
    load_params(g, p.gamma, col, p.cols, p.pvec);
#pragma unroll
    for (int i = 0; i < kLane / 2; ++i) h[k][i] = f2_mul(f2_mul(h[k][i], f2(r, r)), g[i]);
    if (p.beta) {
      load_params(g, p.beta, col, p.cols, p.pvec);
#pragma unroll
      for (int i = 0; i < kLane / 2; ++i) h[k][i] = f2_add(h[k][i], g[i]);
    }
    if (p.silu) silu(h[k]);
    const Fp8Scale q = fp8_scale(team_amax(lane_amax(h[k])));
    const uint4 codes = fp8_codes(h[k], q);
    if (row < p.rows) {
      ok = ok && q.finite;
      if (col < p.pitch) *reinterpret_cast<uint4*>(p.codes + static_cast<int64_t>(row) * p.pitch + col) = codes;
      if (col < p.cols && (threadIdx.x & (kFp8Team - 1)) == 0)
        p.scales[static_cast<int64_t>(col / kFp8Block) * p.rows + row] = q.s;
    }
  }
  if (!ok) raise_fault(p.fault, FAULT_RANGE, 47);
}

// ================================================================================ host side
namespace {

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t size_of(vae_dtype_t t) { return t == VAE_FP32 ? 4 : 2; }
bool value_type(vae_dtype_t t) { return t == VAE_BF16 || t == VAE_FP32; }

vae_status_t fail(vae_status_t code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
vae_status_t fail(vae_status_t code, const char* fmt, ...) {
  char msg[200];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return op_error(code, msg);
}

vae_status_t launched() {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? VAE_OK : fail(VAE_ERR_CUDA, "CUDA error: %s", cudaGetErrorString(e));
}

vae_status_t check_sizes(int64_t rows, int64_t ld, int cols) {
  if (rows < 0 || cols <= 0 || ld < cols)
    return fail(VAE_ERR_INVALID_ARG, "bad sizes: %lld rows, %d columns, row stride %lld", static_cast<long long>(rows), cols,
                static_cast<long long>(ld));
  if (cols > kMaxCols) return fail(VAE_ERR_UNSUPPORTED, "%d columns (at most %d)", cols, kMaxCols);
  if (ld > (int64_t(1) << 32))
    return fail(VAE_ERR_UNSUPPORTED, "row stride %lld (at most 2^32)", static_cast<long long>(ld));
  // (the rows of a thread block past the last one are counted in 32 bits, too)
  if (rows > 0x7fff0000LL || rows > (int64_t(1) << 40) / cols)
    return fail(VAE_ERR_UNSUPPORTED, "%lld x %d values", static_cast<long long>(rows), cols);
  return VAE_OK;
}

vae_status_t check_desc(const vae_fp8_desc_t* d) {
  if (!value_type(d->dtype)) return fail(VAE_ERR_INVALID_ARG, "values are bf16 or fp32");
  if (d->block_rows != 1 && d->block_rows != kFp8Block)
    return fail(VAE_ERR_INVALID_ARG, "blocks of %d rows (1 or %d)", d->block_rows, kFp8Block);
  return check_sizes(d->rows, d->ld, d->cols);
}

// whole: the vectors of a row cover its last block (quantisation)
void fill(Fp8Params& p, const vae_fp8_desc_t* d, const void* values, bool whole) {
  p.rows = static_cast<int>(d->rows);
  p.cols = d->cols;
  p.ld = d->ld;
  p.pitch = (d->cols + 15) / 16 * 16;
  p.row_shift = d->block_rows == 1 ? 0 : 7;
  p.row_blocks = static_cast<int>((d->rows + d->block_rows - 1) / d->block_rows);
  p.vpr = whole ? (d->cols + kFp8Block - 1) / kFp8Block * kFp8Team : (d->cols + kLane - 1) / kLane;
  p.vpr_magic = static_cast<uint32_t>(((1ull << 32) + p.vpr - 1) / p.vpr);
  p.vpr_magic64 = ~uint64_t(0) / p.vpr + 1;  // (2^64 / vpr rounded up, unless vpr is 1)
  p.a32 = aligned(values, 32) && (d->ld * size_of(d->dtype)) % 32 == 0;
  p.fault = fault_word();
}

template <typename T>
void launch_quantize(const Fp8Params& p, bool vec, bool blocks, unsigned grid, cudaStream_t s) {
  if (blocks) {
    if (vec) quantize_fp8_block_kernel<T, true><<<grid, kThreads, 0, s>>>(p);
    else quantize_fp8_block_kernel<T, false><<<grid, kThreads, 0, s>>>(p);
  } else {
    if (vec) quantize_fp8_kernel<T, true><<<grid, kThreads, 0, s>>>(p);
    else quantize_fp8_kernel<T, false><<<grid, kThreads, 0, s>>>(p);
  }
}

// The smallest team whose threads, with two vectors each at most, hold a row (rows of up to 512 columns: one vector each).
template <typename TX, typename TR, bool kVec>
void launch_rms(const Fp8RmsParams& p, cudaStream_t s) {
  const auto teams = [&](int team) { return static_cast<unsigned>((static_cast<int64_t>(p.rows) * team + kThreads - 1) / kThreads); };
  if (p.cols <= 128) {
    residual_rms_fp8_kernel<TX, TR, kVec, 8, 1><<<teams(8), kThreads, 0, s>>>(p);
  } else if (p.cols <= 256) {
    residual_rms_fp8_kernel<TX, TR, kVec, 16, 1><<<teams(16), kThreads, 0, s>>>(p);
  } else if (p.cols <= 512) {
    residual_rms_fp8_kernel<TX, TR, kVec, 32, 1><<<teams(32), kThreads, 0, s>>>(p);
  } else if (p.cols <= 1024) {
    residual_rms_fp8_kernel<TX, TR, kVec, 32, 2><<<teams(32), kThreads, 0, s>>>(p);
  } else {
    constexpr int kVecs = kVec ? 2 : 4;
    const unsigned threads = static_cast<unsigned>((p.cols + 32 * kLane * kVecs - 1) / (32 * kLane * kVecs)) * 32;
    residual_rms_fp8_kernel<TX, TR, kVec, 0, kVecs><<<p.rows, threads, 0, s>>>(p);
  }
}

}  // namespace
}  // namespace vae

using namespace vae;

extern "C" size_t vae_fp8_codes_bytes(int64_t rows, int cols) {
  if (rows < 0 || cols <= 0) return 0;
  return static_cast<size_t>(rows) * ((static_cast<size_t>(cols) + 15) / 16 * 16);
}

extern "C" size_t vae_fp8_scales_bytes(int64_t rows, int cols, int block_rows) {
  if (rows < 0 || cols <= 0 || (block_rows != 1 && block_rows != kFp8Block)) return 0;
  return (static_cast<size_t>(rows) + block_rows - 1) / block_rows * ((static_cast<size_t>(cols) + kFp8Block - 1) / kFp8Block) * 4;
}

extern "C" vae_status_t vae_quantize_fp8(const void* x, void* codes, float* scales, const vae_fp8_desc_t* d, void* stream) {
  if (!d) return fail(VAE_ERR_INVALID_ARG, "null argument");
  vae_status_t st = check_desc(d);
  if (st) return st;
  if (d->rows == 0) return VAE_OK;
  if (!x || !codes || !scales) return fail(VAE_ERR_INVALID_ARG, "null argument");
  const size_t esz = size_of(d->dtype);
  if (!aligned(x, esz) || !aligned(codes, 16) || !aligned(scales, 4))
    return fail(VAE_ERR_ALIGNMENT, "codes must be 16-byte aligned, x and scales aligned to their elements");
  Fp8Params p{};
  fill(p, d, x, true);
  p.x = x;
  p.y = codes;
  p.scales = scales;
  const bool vec = aligned(x, 16) && (d->ld * esz) % 16 == 0;
  const bool blocks = d->block_rows != 1;
  const int64_t grid = blocks ? static_cast<int64_t>(p.row_blocks) * (p.vpr / kFp8Team)
                              : (d->rows * p.vpr + kThreads * kVpt - 1) / (kThreads * kVpt);
  if (grid > 0x7fffffffLL) return fail(VAE_ERR_UNSUPPORTED, "too many values for one call");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d->dtype == VAE_FP32) launch_quantize<float>(p, vec, blocks, static_cast<unsigned>(grid), s);
  else launch_quantize<__nv_bfloat16>(p, vec, blocks, static_cast<unsigned>(grid), s);
  return launched();
}

extern "C" vae_status_t vae_dequantize_fp8(const void* codes, const float* scales, void* y, const vae_fp8_desc_t* d,
                                           void* stream) {
  if (!d) return fail(VAE_ERR_INVALID_ARG, "null argument");
  vae_status_t st = check_desc(d);
  if (st) return st;
  if (d->rows == 0) return VAE_OK;
  if (!codes || !scales || !y) return fail(VAE_ERR_INVALID_ARG, "null argument");
  const size_t esz = size_of(d->dtype);
  if (!aligned(y, esz) || !aligned(codes, 16) || !aligned(scales, 4))
    return fail(VAE_ERR_ALIGNMENT, "codes must be 16-byte aligned, y and scales aligned to their elements");
  Fp8Params p{};
  fill(p, d, y, false);
  p.x = codes;
  p.y = y;
  p.scales = const_cast<float*>(scales);
  const bool vec = aligned(y, 16) && (d->ld * esz) % 16 == 0;
  const int64_t grid = (d->rows * p.vpr + kThreads * kVpt - 1) / (kThreads * kVpt);
  if (grid > 0x7fffffffLL) return fail(VAE_ERR_UNSUPPORTED, "too many values for one call");
  const unsigned g = static_cast<unsigned>(grid);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d->dtype == VAE_FP32) {
    if (vec) dequantize_fp8_kernel<float, true><<<g, kThreads, 0, s>>>(p);
    else dequantize_fp8_kernel<float, false><<<g, kThreads, 0, s>>>(p);
  } else {
    if (vec) dequantize_fp8_kernel<__nv_bfloat16, true><<<g, kThreads, 0, s>>>(p);
    else dequantize_fp8_kernel<__nv_bfloat16, false><<<g, kThreads, 0, s>>>(p);
  }
  return launched();
}

extern "C" vae_status_t vae_gemm_fp8(const void* a_codes, const float* a_scales, const void* b_codes, const float* b_scales,
                                     const float* bias, void* D, const vae_fp8_gemm_desc_t* d, void* stream) {
  if (!d) return fail(VAE_ERR_INVALID_ARG, "null argument");
  if (!value_type(d->out_dtype)) return fail(VAE_ERR_INVALID_ARG, "D is bf16 or fp32");
  if (d->M < 0 || d->N <= 0 || d->K <= 0 || d->ld_d < d->N)
    return fail(VAE_ERR_INVALID_ARG, "bad sizes: M %d, N %d, K %d, row stride %lld", d->M, d->N, d->K,
                static_cast<long long>(d->ld_d));
  if (d->K > kMaxCols || d->N > (1 << 30) || d->M > (1 << 30))
    return fail(VAE_ERR_UNSUPPORTED, "M %d, N %d, K %d (at most 2^30, 2^30, %d)", d->M, d->N, d->K, kMaxCols);
  if (d->ld_d > (int64_t(1) << 32))
    return fail(VAE_ERR_UNSUPPORTED, "row stride %lld (at most 2^32)", static_cast<long long>(d->ld_d));
  if ((static_cast<int64_t>(d->M) + 127) / 128 * ((static_cast<int64_t>(d->N) + 127) / 128) > (1 << 30))
    return fail(VAE_ERR_UNSUPPORTED, "M %d, N %d: more than 2^30 tiles of 128 x 128", d->M, d->N);
  if (d->M == 0) return VAE_OK;
  if (!a_codes || !a_scales || !b_codes || !b_scales || !D) return fail(VAE_ERR_INVALID_ARG, "null argument");
  if (!aligned(a_codes, 16) || !aligned(b_codes, 16) || !aligned(a_scales, 4) || !aligned(b_scales, 4) ||
      !aligned(D, size_of(d->out_dtype)) || (bias && !aligned(bias, 4)))
    return fail(VAE_ERR_ALIGNMENT, "codes must be 16-byte aligned, scales, bias and D aligned to their elements");
  Fp8GemmArgs a{};
  a.M = d->M; a.N = d->N; a.K = d->K; a.alpha = d->alpha;
  a.a_codes = a_codes; a.a_scales = a_scales; a.b_codes = b_codes; a.b_scales = b_scales;
  a.bias = bias; a.y = D; a.out_f32 = d->out_dtype == VAE_FP32; a.ldd = d->ld_d;
  const cudaError_t e = launch_gemm_fp8(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VAE_OK : fail(VAE_ERR_CUDA, "CUDA error: %s", cudaGetErrorString(e));
}

extern "C" vae_status_t vae_residual_rmsnorm_silu_fp8(const void* x, const void* residual, const float* gamma,
                                                      const float* beta, void* total, void* codes, float* scales,
                                                      const vae_fp8_rms_desc_t* d, void* stream) {
  if (!d) return fail(VAE_ERR_INVALID_ARG, "null argument");
  if (!value_type(d->dtype) || !value_type(d->residual_dtype))
    return fail(VAE_ERR_INVALID_ARG, "x, the residual and the total are bf16 or fp32");
  if (!(d->eps >= 0.f)) return fail(VAE_ERR_INVALID_ARG, "eps %g", d->eps);
  vae_status_t st = check_sizes(d->rows, d->ld_x, d->cols);
  if (!st && residual) st = check_sizes(d->rows, d->ld_residual, d->cols);
  if (!st && total) st = check_sizes(d->rows, d->ld_total, d->cols);
  if (st) return st;
  if (d->cols > kRmsMaxCols)
    return fail(VAE_ERR_UNSUPPORTED, "RMS norm over %d columns (at most %d)", d->cols, kRmsMaxCols);
  if (d->rows == 0) return VAE_OK;
  if (!x || !gamma || !codes || !scales) return fail(VAE_ERR_INVALID_ARG, "null argument");
  const size_t ex = size_of(d->dtype), er = size_of(d->residual_dtype);
  if (!aligned(x, ex) || !aligned(residual, er) || !aligned(total, er) || !aligned(gamma, 4) || !aligned(beta, 4) ||
      !aligned(codes, 16) || !aligned(scales, 4))
    return fail(VAE_ERR_ALIGNMENT, "codes must be 16-byte aligned, the other pointers aligned to their elements");
  Fp8RmsParams p{};
  p.x = x; p.residual = residual; p.total = total;
  p.gamma = gamma; p.beta = beta;
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = scales;
  p.ld_x = d->ld_x; p.ld_residual = d->ld_residual; p.ld_total = d->ld_total;
  p.rows = static_cast<int>(d->rows);
  p.cols = d->cols;
  p.pitch = (d->cols + 15) / 16 * 16;
  p.eps = d->eps;
  p.inv_cols = 1.0f / static_cast<float>(d->cols);
  p.silu = d->silu != 0;
  p.ax32 = aligned(x, 32) && (d->ld_x * ex) % 32 == 0;
  p.ar32 = aligned(residual, 32) && (d->ld_residual * er) % 32 == 0;
  p.at32 = aligned(total, 32) && (d->ld_total * er) % 32 == 0;
  p.pvec = aligned(gamma, 16) && aligned(beta, 16);
  p.fault = fault_word();
  const bool vec = aligned(x, 16) && (d->ld_x * ex) % 16 == 0 &&
                   (!residual || (aligned(residual, 16) && (d->ld_residual * er) % 16 == 0)) &&
                   (!total || (aligned(total, 16) && (d->ld_total * er) % 16 == 0));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  using bf16 = __nv_bfloat16;
  const bool xf = d->dtype == VAE_FP32, rf = d->residual_dtype == VAE_FP32;
  if (vec) {
    if (xf && rf) launch_rms<float, float, true>(p, s);
    else if (xf) launch_rms<float, bf16, true>(p, s);
    else if (rf) launch_rms<bf16, float, true>(p, s);
    else launch_rms<bf16, bf16, true>(p, s);
  } else {
    if (xf && rf) launch_rms<float, float, false>(p, s);
    else if (xf) launch_rms<float, bf16, false>(p, s);
    else if (rf) launch_rms<bf16, float, false>(p, s);
    else launch_rms<bf16, bf16, false>(p, s);
  }
  return launched();
}
