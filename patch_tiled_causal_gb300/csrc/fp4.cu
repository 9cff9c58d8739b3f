// Microscaled 4-bit operands: quantisation, reading back, the norms that write them, and the entry points.
//
// TensorRT-LLM PR #16066 "ParallelVAE_TrtllmWan for native Wan VAE" (reviewer comment) names 4-bit
// quantisation with the norm and SiLU fused into it for the Wan VAE; the formats here are the two the tensor cores
// multiply with block scales (kind::mxf4, kind::mxf4nvf4).  The product is in gemm_fp4.cu, the norms' kernels
// in norm.cu next to the ones with wider outputs.
#include <cstdarg>
#include <cstdio>

#include "fp4.cuh"

namespace vae {
namespace {

struct Fp4Params {
  const void* x;        // quantise: values in; read back: codes in
  void* y;              // quantise: codes out; read back: values out
  uint8_t* scales;
  int64_t ld;           // elements between rows of the values
  int rows, cols;
  int pitch;            // bytes between rows of the codes
  int vpr;              // vectors (of 16 columns) handled per row
  uint32_t vpr_magic;   // ceil(2^32 / vpr)
  uint64_t vpr_magic64; // ceil(2^64 / vpr) (vpr >= 2)
  int64_t vecs;         // vectors handled in all
  int groups;           // 4-block scale groups per row tile
  Fp4Scale ts;
  int a32;              // rows of the values start on 32-byte boundaries
  uint32_t* fault;
};

constexpr int kThreads = 256;
constexpr int kVpt = 2;  // vectors of 16 values in flight per thread
constexpr int kMaxCols = 1 << 18;  // a vector index inside a block times vpr stays below 2^32 (vpr_magic)

// First vector of this block -> (row, vector in its row); the block's later vectors then need 32 bits only.
VAE_DEV void block_origin(const Fp4Params& p, int& row0, uint32_t& rem0) {
  const int64_t base = static_cast<int64_t>(blockIdx.x) * (kThreads * kVpt);
  // base / vpr: exact, since base * vpr < 2^64 (a 64-bit division would cost each thread as much as 8 values)
  const int64_t r = p.vpr == 1 ? base : static_cast<int64_t>(__umul64hi(static_cast<uint64_t>(base), p.vpr_magic64));
  row0 = static_cast<int>(r);
  rem0 = static_cast<uint32_t>(base - r * p.vpr);
}

}  // namespace

// One vector of 16 columns per lane and step; the vectors of a row run to the end of its last group of 4
// blocks, and the rows to the end of the last scale tile, so that every byte of the codes' padding and of the
// scale tiles is written (zeros).  HBM-bound by its bytes (x read once, 4.25 (MXFP4) or 4.5 (NVFP4) bits per value
// written), and close to its instructions: 8 values per lane took 22 of them per value and 55 us on 73920 x 1024 bf16 into
// NVFP4; the scale's arithmetic, the addresses and the shuffles fall with the lanes per block.  That round trip, 386 MB,
// takes 65 us, 5.9 TB/s.
// kVec: rows start on 16-byte boundaries; otherwise a warp reads its elements 32 at a time and hands them out through
// shared memory (5003 x 1001 fp32 round trip: each lane on its own elements 34 us, this way 18).
template <int kFmt, typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) quantize_fp4_kernel(const __grid_constant__ Fp4Params p) {
  constexpr int kTeam = kFp4Team<kFmt>;
  int row0;
  uint32_t rem0;
  block_origin(p, row0, rem0);
  const T* x = static_cast<const T*>(p.x);
  const int lane = threadIdx.x & 31;
  int row[kVpt];
  int col[kVpt];
  LaneVec<T> in[kVpt];
#pragma unroll
  for (int k = 0; k < kVpt; ++k) {
    const uint32_t idx = rem0 + static_cast<uint32_t>(k * kThreads) + threadIdx.x;
    const uint32_t r = __umulhi(idx, p.vpr_magic);  // (vpr >= 2 here: a group of 4 blocks)
    row[k] = row0 + static_cast<int>(r);
    col[k] = static_cast<int>(idx - r * static_cast<uint32_t>(p.vpr)) * kLane;
    if constexpr (kVec) {
      in[k].zero();
      if (row[k] < p.rows) {
        const T* src = x + row[k] * p.ld + col[k];
        if (col[k] + kLane <= p.cols) {
          in[k].load(src, p.a32);
        } else {
#pragma unroll
          for (int i = 0; i < kLane; ++i)
            if (col[k] + i < p.cols) reinterpret_cast<T*>(in[k].w)[i] = src[i];
        }
      }
    } else {
      __shared__ __align__(16) T stage[kThreads / 32][32 * kLane];
      T* sh = stage[threadIdx.x >> 5];
      T e[kLane];
#pragma unroll
      for (int i = 0; i < kLane; ++i) {
        int er, ec;
        element_of(i, lane, row[k], col[k], er, ec);
        e[i] = from_f<T>(0.f);
        if (er < p.rows && ec < p.cols) e[i] = x[er * p.ld + ec];
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kLane; ++i) sh[i * 32 + lane] = e[i];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < LaneVec<T>::kW; i += 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(sh + lane * kLane) + i);
        in[k].w[i] = u.x; in[k].w[i + 1] = u.y; in[k].w[i + 2] = u.z; in[k].w[i + 3] = u.w;
      }
    }
  }
  const int last = (p.rows - 1) | 127;  // the last row of the last scale tile
  bool all_ok = true;
#pragma unroll
  for (int k = 0; k < kVpt; ++k) {
    F2 v[kLane / 2];
    in[k].get(v);
    uint2 codes;
    uint32_t byte;
    bool ok;
    fp4_quantize<kFmt>(v, p.ts, codes, byte, ok);
    all_ok = all_ok && ok;
    const uint32_t word = fp4_scale_word<kTeam>(byte, lane);  // (rows and blocks of padding: zeros quantise to byte 0)
    const int r = row[k];
    if (r < p.rows && (col[k] >> 1) < p.pitch)
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.y) + static_cast<int64_t>(r) * p.pitch + (col[k] >> 1)) = codes;
    if (r <= last && (lane & (4 * kTeam - 1)) == 0)
      *reinterpret_cast<uint32_t*>(p.scales + fp4_scale_offset(r, col[k] / kFp4Block<kFmt>, p.groups)) = word;
  }
  if (!all_ok) raise_fault(p.fault, FAULT_RANGE, 40);
}

// Values of packed codes: one vector of 16 columns per lane and step.  HBM-bound like the quantisation.
template <int kFmt, typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) dequantize_fp4_kernel(const __grid_constant__ Fp4Params p) {
  int row0;
  uint32_t rem0;
  block_origin(p, row0, rem0);
  const uint8_t* codes = static_cast<const uint8_t*>(p.x);
  T* y = static_cast<T*>(p.y);
  const int lane = threadIdx.x & 31;
  int row[kVpt];
  int col[kVpt];
  uint2 c[kVpt];
  uint32_t s[kVpt];
#pragma unroll
  for (int k = 0; k < kVpt; ++k) {
    const uint32_t idx = rem0 + static_cast<uint32_t>(k * kThreads) + threadIdx.x;
    const uint32_t q = p.vpr == 1 ? idx : __umulhi(idx, p.vpr_magic);
    col[k] = static_cast<int>(idx - q * static_cast<uint32_t>(p.vpr)) * kLane;
    const int r = row0 + static_cast<int>(q);
    row[k] = r;
    c[k] = make_uint2(0u, 0u);
    s[k] = 0u;
    if (r < p.rows) {
      c[k] = __ldcs(reinterpret_cast<const uint2*>(codes + static_cast<int64_t>(r) * p.pitch + (col[k] >> 1)));
      s[k] = p.scales[fp4_scale_offset(r, col[k] / kFp4Block<kFmt>, p.groups)];
    }
  }
#pragma unroll
  for (int k = 0; k < kVpt; ++k) {
    float v[kLane];
    const float st = fp4_scale_value<kFmt>(s[k]);
    e2m1x8_values(c[k].x, v);
    e2m1x8_values(c[k].y, v + 8);
#pragma unroll
    for (int i = 0; i < kLane; ++i) v[i] = v[i] * st * p.ts.t;
    if constexpr (kVec) {
      if (row[k] >= p.rows) continue;
      T* dst = y + row[k] * p.ld + col[k];
      if (col[k] + kLane <= p.cols) {
        store_lane(dst, v, p.a32);
      } else {
#pragma unroll
        for (int i = 0; i < kLane; ++i)
          if (col[k] + i < p.cols) dst[i] = from_f<T>(v[i]);
      }
    } else {
      __shared__ __align__(16) T stage[kThreads / 32][32 * kLane];
      T* sh = stage[threadIdx.x >> 5];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kLane; i += 8) store8(sh + lane * kLane + i, v + i);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kLane; ++i) {
        int er, ec;
        element_of(i, lane, row[k], col[k], er, ec);
        if (er < p.rows && ec < p.cols) y[er * p.ld + ec] = sh[i * 32 + lane];
      }
    }
  }
}

namespace {

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int block_of(int format) { return format == VAE_MXFP4 ? 32 : 16; }

vae_status_t fail(vae_status_t code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
vae_status_t fail(vae_status_t code, const char* fmt, ...) {
  char msg[200];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return op_error(code, msg);
}

vae_status_t check_format(int format, float ts) {
  if (format != VAE_MXFP4 && format != VAE_NVFP4) return fail(VAE_ERR_INVALID_ARG, "unknown 4-bit format %d", format);
  if (format == VAE_MXFP4 && ts != 1.0f)
    return fail(VAE_ERR_INVALID_ARG, "MXFP4 has no tensor scale (got %g, must be 1)", ts);
  if (!(ts >= 0x1p-64f && ts <= 0x1p64f))
    return fail(VAE_ERR_INVALID_ARG, "tensor scale %g outside 2^-64 .. 2^64", ts);
  return VAE_OK;
}

vae_status_t check_desc(const vae_fp4_desc_t* d) {
  vae_status_t st = check_format(d->format, d->tensor_scale);
  if (st) return st;
  if (d->dtype != VAE_BF16 && d->dtype != VAE_FP32) return fail(VAE_ERR_INVALID_ARG, "values are bf16 or fp32");
  if (d->rows < 0 || d->cols <= 0 || d->ld < d->cols)
    return fail(VAE_ERR_INVALID_ARG, "bad sizes: %lld rows, %d columns, row stride %lld", static_cast<long long>(d->rows),
                d->cols, static_cast<long long>(d->ld));
  if (d->cols > kMaxCols) return fail(VAE_ERR_UNSUPPORTED, "%d columns (at most %d)", d->cols, kMaxCols);
  if (d->ld > (int64_t(1) << 32))
    return fail(VAE_ERR_UNSUPPORTED, "row stride %lld (at most 2^32)", static_cast<long long>(d->ld));
  // (the rows of the last scale tile and of a block's vectors past it are counted in 32 bits, too)
  if (d->rows > 0x7fff0000LL || d->rows > (int64_t(1) << 40) / d->cols)
    return fail(VAE_ERR_UNSUPPORTED, "%lld x %d values", static_cast<long long>(d->rows), d->cols);
  return VAE_OK;
}

// Common part of the two directions; whole_tiles: cover the padding too (quantisation).
void fill(Fp4Params& p, const vae_fp4_desc_t* d, bool whole_tiles) {
  const int blk = block_of(d->format);
  p.rows = static_cast<int>(d->rows);
  p.cols = d->cols;
  p.ld = d->ld;
  p.pitch = (d->cols + 31) / 32 * 16;
  p.groups = fp4_groups(d->format, d->cols);
  p.vpr = whole_tiles ? p.groups * 4 * blk / kLane : (d->cols + kLane - 1) / kLane;
  p.vpr_magic = static_cast<uint32_t>(((1ull << 32) + p.vpr - 1) / p.vpr);
  p.vpr_magic64 = ~uint64_t(0) / p.vpr + 1;  // (2^64 / vpr rounded up, unless vpr is 1)
  p.vecs = (whole_tiles ? (d->rows + 127) / 128 * 128 : d->rows) * p.vpr;
  p.ts = fp4_scale(d->tensor_scale);
  p.fault = fault_word();
}

template <int kFmt, typename T>
void launch_quantize(const Fp4Params& p, bool vec, unsigned blocks, cudaStream_t s) {
  if (vec) quantize_fp4_kernel<kFmt, T, true><<<blocks, kThreads, 0, s>>>(p);
  else quantize_fp4_kernel<kFmt, T, false><<<blocks, kThreads, 0, s>>>(p);
}
template <int kFmt, typename T>
void launch_dequantize(const Fp4Params& p, bool vec, unsigned blocks, cudaStream_t s) {
  if (vec) dequantize_fp4_kernel<kFmt, T, true><<<blocks, kThreads, 0, s>>>(p);
  else dequantize_fp4_kernel<kFmt, T, false><<<blocks, kThreads, 0, s>>>(p);
}

}  // namespace
}  // namespace vae

using namespace vae;

extern "C" size_t vae_fp4_codes_bytes(int64_t rows, int cols) {
  if (rows < 0 || cols <= 0) return 0;
  return static_cast<size_t>(rows) * ((static_cast<size_t>(cols) + 31) / 32 * 16);
}

extern "C" size_t vae_fp4_scales_bytes(vae_fp4_format_t format, int64_t rows, int cols) {
  if ((format != VAE_MXFP4 && format != VAE_NVFP4) || rows < 0 || cols <= 0) return 0;
  const size_t blk = static_cast<size_t>(block_of(format));
  const size_t groups = ((static_cast<size_t>(cols) + blk - 1) / blk + 3) / 4;
  return (static_cast<size_t>(rows) + 127) / 128 * groups * 512;
}

extern "C" vae_status_t vae_quantize_fp4(const void* x, void* codes, void* scales, const vae_fp4_desc_t* d,
                                         void* stream) {
  if (!d) return fail(VAE_ERR_INVALID_ARG, "null argument");
  vae_status_t st = check_desc(d);
  if (st) return st;
  if (d->rows == 0) return VAE_OK;
  if (!x || !codes || !scales) return fail(VAE_ERR_INVALID_ARG, "null argument");
  const size_t esz = d->dtype == VAE_FP32 ? 4 : 2;
  if (!aligned(x, esz) || !aligned(codes, 16) || !aligned(scales, 16))
    return fail(VAE_ERR_ALIGNMENT, "codes and scales must be 16-byte aligned, x aligned to its elements");
  Fp4Params p{};
  fill(p, d, true);
  p.x = x;
  p.a32 = aligned(x, 32) && (d->ld * esz) % 32 == 0;
  p.y = codes;
  p.scales = static_cast<uint8_t*>(scales);
  const bool vec = aligned(x, 16) && (d->ld * esz) % 16 == 0;
  const int64_t blocks = (p.vecs + kThreads * kVpt - 1) / (kThreads * kVpt);
  if (blocks > 0x7fffffffLL) return fail(VAE_ERR_UNSUPPORTED, "too many values for one call");
  const unsigned nb = static_cast<unsigned>(blocks);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d->format == VAE_MXFP4) {
    if (d->dtype == VAE_FP32) launch_quantize<VAE_MXFP4, float>(p, vec, nb, s);
    else launch_quantize<VAE_MXFP4, __nv_bfloat16>(p, vec, nb, s);
  } else {
    if (d->dtype == VAE_FP32) launch_quantize<VAE_NVFP4, float>(p, vec, nb, s);
    else launch_quantize<VAE_NVFP4, __nv_bfloat16>(p, vec, nb, s);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? VAE_OK : fail(VAE_ERR_CUDA, "CUDA error: %s", cudaGetErrorString(e));
}

extern "C" vae_status_t vae_dequantize_fp4(const void* codes, const void* scales, void* y, const vae_fp4_desc_t* d,
                                           void* stream) {
  if (!d) return fail(VAE_ERR_INVALID_ARG, "null argument");
  vae_status_t st = check_desc(d);
  if (st) return st;
  if (d->rows == 0) return VAE_OK;
  if (!codes || !scales || !y) return fail(VAE_ERR_INVALID_ARG, "null argument");
  const size_t esz = d->dtype == VAE_FP32 ? 4 : 2;
  if (!aligned(y, esz) || !aligned(codes, 16) || !aligned(scales, 16))
    return fail(VAE_ERR_ALIGNMENT, "codes and scales must be 16-byte aligned, y aligned to its elements");
  Fp4Params p{};
  fill(p, d, false);
  p.x = codes;
  p.a32 = aligned(y, 32) && (d->ld * esz) % 32 == 0;
  p.y = y;
  p.scales = static_cast<uint8_t*>(const_cast<void*>(scales));
  const bool vec = aligned(y, 16) && (d->ld * esz) % 16 == 0;
  const int64_t blocks = (p.vecs + kThreads * kVpt - 1) / (kThreads * kVpt);
  if (blocks > 0x7fffffffLL) return fail(VAE_ERR_UNSUPPORTED, "too many values for one call");
  const unsigned nb = static_cast<unsigned>(blocks);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d->format == VAE_MXFP4) {
    if (d->dtype == VAE_FP32) launch_dequantize<VAE_MXFP4, float>(p, vec, nb, s);
    else launch_dequantize<VAE_MXFP4, __nv_bfloat16>(p, vec, nb, s);
  } else {
    if (d->dtype == VAE_FP32) launch_dequantize<VAE_NVFP4, float>(p, vec, nb, s);
    else launch_dequantize<VAE_NVFP4, __nv_bfloat16>(p, vec, nb, s);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? VAE_OK : fail(VAE_ERR_CUDA, "CUDA error: %s", cudaGetErrorString(e));
}

extern "C" vae_status_t vae_gemm_fp4(const void* a_codes, const void* a_scales, const void* b_codes,
                                     const void* b_scales, const float* bias, void* D, const vae_fp4_gemm_desc_t* d,
                                     void* stream) {
  if (!d) return fail(VAE_ERR_INVALID_ARG, "null argument");
  vae_status_t st = check_format(d->format, 1.0f);
  if (st) return st;
  if (d->out_dtype != VAE_BF16 && d->out_dtype != VAE_FP32) return fail(VAE_ERR_INVALID_ARG, "D is bf16 or fp32");
  if (d->M < 0 || d->N <= 0 || d->K <= 0 || d->ld_d < d->N)
    return fail(VAE_ERR_INVALID_ARG, "bad sizes: M %d, N %d, K %d, row stride %lld", d->M, d->N, d->K,
                static_cast<long long>(d->ld_d));
  if (d->K > kMaxCols || d->N > (1 << 30) || d->M > (1 << 30))
    return fail(VAE_ERR_UNSUPPORTED, "M %d, N %d, K %d (at most 2^30, 2^30, %d)", d->M, d->N, d->K, kMaxCols);
  if (d->ld_d > (int64_t(1) << 32))
    return fail(VAE_ERR_UNSUPPORTED, "row stride %lld (at most 2^32)", static_cast<long long>(d->ld_d));
  if ((static_cast<int64_t>(d->M) + 255) / 256 * ((static_cast<int64_t>(d->N) + 255) / 256) > (1 << 30))
    return fail(VAE_ERR_UNSUPPORTED, "M %d, N %d: more than 2^30 tiles of 256 x 256", d->M, d->N);
  if (d->M == 0) return VAE_OK;
  if (!a_codes || !a_scales || !b_codes || !b_scales || !D) return fail(VAE_ERR_INVALID_ARG, "null argument");
  if (!aligned(a_codes, 16) || !aligned(a_scales, 16) || !aligned(b_codes, 16) || !aligned(b_scales, 16) ||
      !aligned(D, d->out_dtype == VAE_FP32 ? 4 : 2) || (bias && !aligned(bias, 4)))
    return fail(VAE_ERR_ALIGNMENT, "codes and scales must be 16-byte aligned, bias and D aligned to their elements");
  Fp4GemmArgs a{};
  a.M = d->M; a.N = d->N; a.K = d->K; a.format = d->format; a.alpha = d->alpha;
  a.a_codes = a_codes; a.a_scales = a_scales; a.b_codes = b_codes; a.b_scales = b_scales;
  a.bias = bias; a.y = D; a.out_f32 = d->out_dtype == VAE_FP32; a.ldd = d->ld_d;
  const cudaError_t e = launch_gemm_fp4(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VAE_OK : fail(VAE_ERR_CUDA, "CUDA error: %s", cudaGetErrorString(e));
}

extern "C" vae_status_t vae_patch_groupnorm_silu_fp4(const void* x, const float* gamma, const float* beta, void* codes,
                                                     void* scales, void* workspace, const vae_gn_desc_t* d,
                                                     vae_fp4_format_t format, float tensor_scale, void* stream) {
  if (!x || !gamma || !beta || !codes || !scales || !workspace || !d) return fail(VAE_ERR_INVALID_ARG, "null argument");
  if (!aligned(workspace, 16) || !aligned(scales, 16))
    return fail(VAE_ERR_ALIGNMENT, "pointers must be 16-byte aligned");
  vae_status_t st = check_format(format, tensor_scale);
  vae_gn_desc_t dd = *d;
  dd.out_dtype = VAE_BF16;  // (ignored: the output is the operand)
  if (!st) st = validate_gn_desc(x, codes, &dd);
  if (st) return st;
  if (d->C % 32) return fail(VAE_ERR_UNSUPPORTED, "4-bit operands need C %% 32 == 0 (got %d)", d->C);
  if (static_cast<int64_t>(d->B) * d->T > 65535)
    return fail(VAE_ERR_UNSUPPORTED, "%d x %d frames (at most 65535)", d->B, d->T);
  if (static_cast<double>(d->B) * d->T * d->H * d->W >= 1073741824.0)
    return fail(VAE_ERR_UNSUPPORTED, "%d x %d x %d x %d pixels (below 2^30)", d->B, d->T, d->H, d->W);
  GnArgs g{};
  g.B = d->B; g.T = d->T; g.H = d->H; g.W = d->W; g.C = d->C; g.groups = d->groups; g.eps = d->eps; g.silu = d->silu;
  g.nph = d->n_patch_h; g.npw = d->n_patch_w; g.ph_edges = d->patch_h_edges; g.pw_edges = d->patch_w_edges;
  g.x = x; g.x_f32 = d->in_dtype == VAE_FP32; g.y = codes;
  g.gamma = gamma; g.beta = beta; g.partials = workspace;
  g.fp4 = 1; g.fp4_format = format; g.fp4_scales = scales; g.fp4_ts = tensor_scale;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_gn_fp4(g, s);
  return e == cudaSuccess ? VAE_OK : fail(VAE_ERR_CUDA, "CUDA error: %s", cudaGetErrorString(e));
}

extern "C" vae_status_t vae_channel_rmsnorm_silu_fp4(const void* x, const float* gamma, const float* beta, void* codes,
                                                     void* scales, const vae_rms_desc_t* d, vae_fp4_format_t format,
                                                     float tensor_scale, void* stream) {
  if (!x || !gamma || !beta || !codes || !scales || !d) return fail(VAE_ERR_INVALID_ARG, "null argument");
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(gamma, 32) || !aligned(beta, 32))
    return fail(VAE_ERR_ALIGNMENT, "x, codes, scales must be 16-byte and gamma, beta 32-byte aligned");
  vae_status_t st = check_format(format, tensor_scale);
  if (st) return st;
  if (d->B <= 0 || d->T <= 0 || d->H <= 0 || d->W <= 0 || d->C <= 0 || !(d->eps >= 0.f))
    return fail(VAE_ERR_INVALID_ARG, "bad RMS-norm descriptor");
  if (d->in_dtype != VAE_BF16 && d->in_dtype != VAE_FP32) return fail(VAE_ERR_INVALID_ARG, "bad dtype");
  if (!rms_supported(d->C) || d->C % 32)
    return fail(VAE_ERR_UNSUPPORTED, "RMS norm over %d channels into 4-bit operands not supported", d->C);
  if (static_cast<double>(d->B) * d->T * d->H * d->W >= 1073741824.0)
    return fail(VAE_ERR_UNSUPPORTED, "%d x %d x %d x %d pixels (below 2^30)", d->B, d->T, d->H, d->W);
  GnArgs g{};
  g.B = d->B; g.T = d->T; g.H = d->H; g.W = d->W; g.C = d->C; g.eps = d->eps; g.silu = d->silu;
  g.x = x; g.x_f32 = d->in_dtype == VAE_FP32; g.y = codes;
  g.gamma = gamma; g.beta = beta;
  g.fp4 = 1; g.fp4_format = format; g.fp4_scales = scales; g.fp4_ts = tensor_scale;
  const cudaError_t e = launch_rms(g, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? VAE_OK : fail(VAE_ERR_CUDA, "CUDA error: %s", cudaGetErrorString(e));
}
