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
// vectors of 16 values in flight per thread (quantised with 1 or 2: 73920 x 1024 bf16 35.9, 36.5 us, 3000 x 1024 2.7, 3.0;
// reading back with 1 or 2 is equal to within 1%)
constexpr int kVptIn = 1, kVptOut = 2;
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
  int vpr;               // vectors (of 16 columns), or blocks, handled per row
  uint32_t vpr_magic;    // ceil(2^32 / vpr)
  uint64_t vpr_magic64;  // ceil(2^64 / vpr) (vpr >= 2)
  int a32;               // rows of the values start on 32-byte boundaries
  uint32_t* fault;
};

// First vector of this block -> (row, vector in its row); the block's later vectors then need 32 bits only.
template <int kVpt>
VAE_DEV void block_origin(const Fp8Params& p, int& row0, uint32_t& rem0) {
  const int64_t base = static_cast<int64_t>(blockIdx.x) * (kThreads * kVpt);
  const int64_t r = p.vpr == 1 ? base : static_cast<int64_t>(__umul64hi(static_cast<uint64_t>(base), p.vpr_magic64));
  row0 = static_cast<int>(r);
  rem0 = static_cast<uint32_t>(base - r * p.vpr);
}

// Matrices whose rows start on 16-byte boundaries are read and written 16 values (a vector) per lane.
// The vector at (row, col) of a matrix of rows x cols values, zeros outside it.
template <typename T>
VAE_DEV void load_vec(LaneVec<T>& in, const T* x, int64_t ld, int rows, int cols, int row, int col, bool a32) {
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
}
template <typename T>
VAE_DEV void store_vec(T* y, const float* v, int64_t ld, int rows, int cols, int row, int col, bool a32) {
  if (row >= rows || col >= cols) return;
  T* dst = y + row * ld + col;
  if (col + kLane <= cols) {
    store_lane(dst, v, a32);
  } else {
#pragma unroll
    for (int i = 0; i < kLane; ++i)
      if (col + i < cols) dst[i] = from_f<T>(v[i]);
  }
}

// Rows that start anywhere go 4 adjacent values per lane, a warp per 128 columns, in the widest accesses that their
// alignment allows: 8 bytes, 4, or (bf16 off 4 bytes) 2, 4 and 2; `n` of the 4 values exist.  What the loads bring is kept
// as it is until all of a thread's loads are on their way.
// (16 values per lane, handed out through shared memory, took 22.5 us for 5003 x 1001 fp32 both ways.)
template <typename T> struct Piece;
template <> struct Piece<float> {
  float v[4];
  VAE_DEV void load(const float* p, int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = 0.f;
    if (n >= 4 && (reinterpret_cast<uintptr_t>(p) & 7) == 0) {
      const float2 a = *reinterpret_cast<const float2*>(p), b = *reinterpret_cast<const float2*>(p + 2);
      v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) v[i] = p[i];
    }
  }
  VAE_DEV void get(float* t) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = v[i];
  }
};
template <> struct Piece<__nv_bfloat16> {
  uint32_t w[3];
  bool odd;  // a value, a word, a value (else two words)
  VAE_DEV void load(const __nv_bfloat16* p, int n) {
    const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
    const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 7u;  // (the same for a row's pieces)
    odd = n < 4 || (at & 2u);
    w[0] = w[1] = w[2] = 0u;
    if (n >= 4) {
      if (at == 0u) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        w[0] = u.x; w[1] = u.y;
      } else if (at == 4u) {
        w[0] = reinterpret_cast<const uint32_t*>(p)[0];
        w[1] = reinterpret_cast<const uint32_t*>(p)[1];
      } else {
        w[0] = h[0];
        w[1] = *reinterpret_cast<const uint32_t*>(p + 1);
        w[2] = h[3];
      }
    } else if (n > 0) {
      w[0] = h[0];
      if (n > 1) w[1] = h[1];
      if (n > 2) w[1] |= static_cast<uint32_t>(h[2]) << 16;
    }
  }
  VAE_DEV void get(float* t) const {
    const auto lo = [](uint32_t u) { return __uint_as_float(u << 16); };
    const auto hi = [](uint32_t u) { return __uint_as_float(u & 0xffff0000u); };
    t[0] = lo(w[0]);
    t[1] = odd ? lo(w[1]) : hi(w[0]);
    t[2] = odd ? hi(w[1]) : lo(w[1]);
    t[3] = odd ? lo(w[2]) : hi(w[1]);
  }
};
VAE_DEV void store4(float* p, int n, const float* v) {
  const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p));
  if (n >= 4 && (at & 7u) == 0u) {
    *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    *reinterpret_cast<float2*>(p + 2) = make_float2(v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = v[i];
  }
}
VAE_DEV void store4(__nv_bfloat16* p, int n, const float* v) {
  const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p));
  if (n >= 4) {
    if ((at & 3u) == 0u) {
      __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
      if ((at & 7u) == 0u) {
        *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
      } else {
        reinterpret_cast<__nv_bfloat162*>(p)[0] = a;
        reinterpret_cast<__nv_bfloat162*>(p)[1] = b;
      }
    } else {
      p[0] = f2bf(v[0]);
      *reinterpret_cast<__nv_bfloat162*>(p + 1) = __floats2bfloat162_rn(v[1], v[2]);
      p[3] = f2bf(v[3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = f2bf(v[i]);
  }
}
// max|x| of a lane's 4 values, NaN when any is NaN
VAE_DEV float amax4(const float* v) { return max_abs_or_nan(max_abs_or_nan(v[0], v[1], v[2]), v[3], 0.f); }

// The scales of the four blocks that a warp holds 4 values per lane of, from each lane's maxima m: the lanes 8 b .. 8 b + 7
// find the maximum of block b and its scale, once, and hand it to the others.  s: the scale itself, of block lane / 8.
// (Each lane finding every block's scale by itself takes about 40 instructions for 4 values.)
VAE_DEV void warp_scales4(const float* m, Fp8Scale* q, float& s) {
  const int lane = threadIdx.x & 31;
  const bool h16 = lane & 16, h8 = lane & 8;
  const float a0 = __shfl_xor_sync(0xffffffffu, h16 ? m[0] : m[2], 16), a1 = __shfl_xor_sync(0xffffffffu, h16 ? m[1] : m[3], 16);
  const float k0 = max_abs_or_nan(h16 ? m[2] : m[0], a0, 0.f), k1 = max_abs_or_nan(h16 ? m[3] : m[1], a1, 0.f);
  float v = max_abs_or_nan(h8 ? k1 : k0, __shfl_xor_sync(0xffffffffu, h8 ? k0 : k1, 8), 0.f);
#pragma unroll
  for (int d = 4; d >= 1; d /= 2) v = max_abs_or_nan(v, __shfl_xor_sync(0xffffffffu, v, d), 0.f);
  const Fp8Scale mine = fp8_scale(v);
  const uint32_t finite = __ballot_sync(0xffffffffu, mine.finite), tiny = __ballot_sync(0xffffffffu, mine.k != 1.0f);
  s = mine.s;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    q[b].nsk = __shfl_sync(0xffffffffu, mine.nsk, 8 * b);
    q[b].r = __shfl_sync(0xffffffffu, mine.r, 8 * b);
    q[b].k = (tiny >> (8 * b)) & 1u ? 0x1p64f : 1.0f;
    q[b].finite = (finite >> (8 * b)) & 1u;
  }
}
VAE_DEV uint32_t fp8_codes4(const float* v, const Fp8Scale& q) {
  if (!q.finite) return 0u;
  const F2 nsk = f2(q.nsk, q.nsk), r = f2(q.r, q.r);
  F2 a = f2(v[0], v[1]), b = f2(v[2], v[3]);
  if (q.k != 1.0f) {
    a = f2_mul(a, f2(q.k, q.k));
    b = f2_mul(b, f2(q.k, q.k));
  }
  return e4m3x4(div_by(a, nsk, r), div_by(b, nsk, r));
}

constexpr int kUnits = 4;  // blocks of 128 columns in flight per warp

// Unit u of this warp, of the grid's 128-column pieces of rows -> (row, column block).
VAE_DEV void unit_of(const Fp8Params& p, int u, int& row, int& cb) {
  const int64_t base = static_cast<int64_t>(blockIdx.x) * (kThreads / 32 * kUnits);
  const int64_t r = p.vpr == 1 ? base : static_cast<int64_t>(__umul64hi(static_cast<uint64_t>(base), p.vpr_magic64));
  const uint32_t idx = static_cast<uint32_t>(base - r * p.vpr) + static_cast<uint32_t>(u * (kThreads / 32)) + (threadIdx.x >> 5);
  const uint32_t q = p.vpr == 1 ? idx : __umulhi(idx, p.vpr_magic);
  row = static_cast<int>(r) + static_cast<int>(q);
  cb = static_cast<int>(idx - q * static_cast<uint32_t>(p.vpr));
}

}  // namespace

// One scale per 128 columns of a row.  One vector of 16 columns per lane and step, 8 lanes per block; the vectors of a
// row run to the end of its last block.  HBM-bound by its bytes (x read once, 1 + 1/32 bytes per value written):
// 73920 x 1024 bf16 36.3 us, 6.3 TB/s (68% of the issue slots); fp32 54.0, 7.0 TB/s.
template <typename T>
__global__ void __launch_bounds__(kThreads) quantize_fp8_kernel(const __grid_constant__ Fp8Params p) {
  constexpr int kVpt = kVptIn;
  int row0;
  uint32_t rem0;
  block_origin<kVpt>(p, row0, rem0);
  int row[kVpt], col[kVpt];
  LaneVec<T> in[kVpt];
#pragma unroll
  for (int k = 0; k < kVpt; ++k) {
    const uint32_t idx = rem0 + static_cast<uint32_t>(k * kThreads) + threadIdx.x;
    const uint32_t r = __umulhi(idx, p.vpr_magic);  // (vpr >= 8 here)
    row[k] = row0 + static_cast<int>(r);
    col[k] = static_cast<int>(idx - r * static_cast<uint32_t>(p.vpr)) * kLane;
    load_vec(in[k], static_cast<const T*>(p.x), p.ld, p.rows, p.cols, row[k], col[k], p.a32);
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

// The same for rows that start anywhere; p.vpr counts blocks.  Bound by issue: an access brings 2 - 8 bytes, where a
// vector's brings 16.  40013 x 333 bf16 17.6 us, 2.3 TB/s; 5003 x 1001 fp32 6.4.
template <typename T>
__global__ void __launch_bounds__(kThreads) quantize_fp8_any_kernel(const __grid_constant__ Fp8Params p) {
  const int lane = threadIdx.x & 31;
  int row[kUnits], cb[kUnits];
  Piece<T> in[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    unit_of(p, u, row[u], cb[u]);
    const int col = cb[u] * kFp8Block + lane * 4;
    in[u].load(static_cast<const T*>(p.x) + row[u] * p.ld + col, row[u] < p.rows ? p.cols - col : 0);
  }
  float v[kUnits][4], m[kUnits], s;
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    in[u].get(v[u]);
    m[u] = amax4(v[u]);
  }
  Fp8Scale q[kUnits];
  warp_scales4(m, q, s);
  bool ok = true;
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    if (row[u] >= p.rows) continue;
    ok = ok && q[u].finite;
    const int col = cb[u] * kFp8Block + lane * 4;
    if (col < p.pitch)
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.y) + static_cast<int64_t>(row[u]) * p.pitch + col) = fp8_codes4(v[u], q[u]);
    if (lane == 8 * u) p.scales[static_cast<int64_t>(cb[u]) * p.row_blocks + row[u]] = s;
  }
  if (!ok) raise_fault(p.fault, FAULT_RANGE, 45);
}

// One scale per 128 columns of 128 rows: a thread block per block of values, which stays in registers (64 values a
// thread) between its maximum and its codes.  HBM-bound while blocks start and end unevenly (three per SM): 4096 x 4096
// fp32 16.1 us, 5.2 TB/s.  Rows that start anywhere: 5003 x 1001 fp32 6.8 us, 3.7 TB/s, bf16 9.0, 1.7 (issue, and few
// bytes spilled).
template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads, 3) quantize_fp8_block_kernel(const __grid_constant__ Fp8Params p) {
  // a lane's pieces: kN values each (a vector, or 4 where rows start anywhere), of rows kStep apart
  constexpr int kN = kVec ? kLane : 4, kRow = kFp8Block / kN, kStep = kThreads / kRow, kV = kFp8Block / kStep;
  const int nc = p.vpr;  // column blocks
  const int rb = blockIdx.x / nc, cb = blockIdx.x - rb * nc;
  const int row = rb * kFp8Block + threadIdx.x / kRow, col = cb * kFp8Block + threadIdx.x % kRow * kN;
  F2 v[kV][kN / 2];
  if constexpr (kVec) {
    LaneVec<T> in[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i)
      load_vec(in[i], static_cast<const T*>(p.x), p.ld, p.rows, p.cols, row + i * kStep, col, p.a32);
#pragma unroll
    for (int i = 0; i < kV; ++i) in[i].get(v[i]);
  } else {
    Piece<T> in[kV];
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int r = row + i * kStep;
      in[i].load(static_cast<const T*>(p.x) + r * p.ld + col, r < p.rows ? p.cols - col : 0);
    }
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      float t[4];
      in[i].get(t);
      v[i][0] = f2(t[0], t[1]);
      v[i][1] = f2(t[2], t[3]);
    }
  }
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < kV; ++i)
#pragma unroll
    for (int j = 0; j < kN / 2; ++j) {
      const float2 t = f2_get(v[i][j]);
      m = max_abs_or_nan(m, t.x, t.y);
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
    uint8_t* dst = static_cast<uint8_t*>(p.y) + static_cast<int64_t>(r) * p.pitch + col;
    if constexpr (kVec) {
      *reinterpret_cast<uint4*>(dst) = fp8_codes(v[i], q);
    } else {
      const float2 a = f2_get(v[i][0]), b = f2_get(v[i][1]);
      const float t[4] = {a.x, a.y, b.x, b.y};
      *reinterpret_cast<uint32_t*>(dst) = fp8_codes4(t, q);
    }
  }
  if (threadIdx.x == 0) {
    p.scales[static_cast<int64_t>(cb) * p.row_blocks + rb] = q.s;
    if (!q.finite) raise_fault(p.fault, FAULT_RANGE, 46);
  }
}

// Values of codes: one vector of 16 columns per lane and step.  HBM-bound like the quantisation: 73920 x 1024 bf16
// 34.7 us, 6.5 TB/s.
template <typename T>
__global__ void __launch_bounds__(kThreads) dequantize_fp8_kernel(const __grid_constant__ Fp8Params p) {
  constexpr int kVpt = kVptOut;
  int row0;
  uint32_t rem0;
  block_origin<kVpt>(p, row0, rem0);
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
    store_vec(static_cast<T*>(p.y), v, p.ld, p.rows, p.cols, row[k], col[k], p.a32);
  }
}

// The same for rows that start anywhere, bound by issue: 40013 x 333 bf16 11.9 us, 3.4 TB/s.
template <typename T>
__global__ void __launch_bounds__(kThreads) dequantize_fp8_any_kernel(const __grid_constant__ Fp8Params p) {
  const int lane = threadIdx.x & 31;
  int row[kUnits], col[kUnits];
  uint32_t c[kUnits];
  float s[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    int cb;
    unit_of(p, u, row[u], cb);
    col[u] = cb * kFp8Block + lane * 4;
    c[u] = 0u;
    s[u] = 0.f;
    if (row[u] < p.rows && col[u] < p.cols) {
      c[u] = __ldcs(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.x) +
                                                      static_cast<int64_t>(row[u]) * p.pitch + col[u]));
      s[u] = __ldg(p.scales + static_cast<int64_t>(cb) * p.row_blocks + (row[u] >> p.row_shift));
    }
  }
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    if (row[u] >= p.rows || col[u] >= p.cols) continue;
    float v[4];
    e4m3x4_values(c[u], v);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] *= s[u];
    store4(static_cast<T*>(p.y) + row[u] * p.ld + col[u], p.cols - col[u], v);
  }
}

// ================================================================================ RMS norm of a residual sum
namespace {
constexpr int kRmsMaxCols = 32768;  // 2048 vectors: four for each of 512 threads
// threads of a block that holds one row, and blocks per SM that the compiler leaves registers for
template <int kVecs> constexpr int kRowThreads = kVecs == 2 ? 384 : 512;
// (bf16 alone takes 4 blocks of 256 threads: 140000 x 512 82 us, with 3 95; with fp32 values 4 spill: 73920 x 1024 127, 142.
// Two vectors of bf16 a lane spill with 4 too, 154 bytes a thread, 14 with kept parameters: 100000 x 768 91 us, with 3 103, but 73920 x
// 1024 87.6, 85.9, 15000 x 1024 23.4, 21.7, 3000 x 1024 6.3, 5.9.  Among the others two forms spill much, both of fp32 alone:
// four vectors, 174 bytes, and 16 blocks a warp of rows that start anywhere, 124.)
template <typename TX, typename TR, int kTeam, int kVecs>
constexpr int kRmsBlocks = kTeam ? (sizeof(TX) + sizeof(TR) == 4 ? 4 : 3) : kVecs == 2 ? 2 : 1;

struct Fp8RmsParams {
  const void* x; const void* residual; void* total;  // residual, total: may be null
  const float* gamma; const float* beta;             // beta: may be null
  uint8_t* codes; float* scales;
  int64_t ld_x, ld_residual, ld_total;
  int rows, cols, pitch;
  float eps, inv_cols;
  int silu;
  int ax32, ar32, at32;  // rows of x, the residual, the total start on 32-byte boundaries
  int pvec;              // gamma and beta are 32-byte aligned
  uint32_t* fault;
};

// 16 parameters from col on, zeros behind the last column; vec: src is 32-byte aligned (32-byte loads: a warp's fill the
// L1 cache's pipe half as long as 16-byte ones)
VAE_DEV void load_params(F2* v, const float* src, int col, int cols, bool vec) {
  if (vec && col + kLane <= cols) {
    LaneVec<float> in;
    in.load(src + col, true);
    in.get(v);
  } else {
#pragma unroll
    for (int i = 0; i < kLane / 2; ++i)
      v[i] = f2(col + 2 * i < cols ? __ldg(src + col + 2 * i) : 0.f,
                col + 2 * i + 1 < cols ? __ldg(src + col + 2 * i + 1) : 0.f);
  }
}

// 1 / sqrt(mean + eps) of a row, NaN where the sum of squares is not finite
VAE_DEV float inverse_rms(const Fp8RmsParams& p, float ss) {
  return ss <= 3.402823466e38f ? __frcp_rn(__fsqrt_rn(fmaf(ss, p.inv_cols, p.eps))) : __int_as_float(0x7fffffff);
}

// Squares are rounded to multiples of 2^-149, which counts where mean + eps is small.  In calls with an eps below kTinyMean
// (kernels of their own, kTiny: the others keep their registers) such a row, whose values are below 2^-42, is multiplied by 2^96 and
// summed up once more, against eps * 2^192.
constexpr float kTinyMean = 0x1p-100f, kTinyScale = 0x1p96f;
VAE_DEV bool tiny_mean(const Fp8RmsParams& p, float ss) { return fmaf(ss, p.inv_cols, p.eps) < kTinyMean; }
VAE_DEV float inverse_rms_scaled(const Fp8RmsParams& p, float ss) {
  return __frcp_rn(__fsqrt_rn(fmaf(ss, p.inv_cols, p.eps * kTinyScale * kTinyScale)));
}

// The sum of the warps' sums, in the order of the warps; `part`: 32 floats that no earlier call of the last two used.
VAE_DEV float block_sum(float ss, float* part) {
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ss;
  __syncthreads();
  ss = 0.f;
  for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) ss += part[i];
  return ss;
}
}  // namespace

// h = x + residual (fp32), total = h rounded, y = SiLU(h / sqrt(mean h^2 + eps) * gamma + beta), y quantised with one
// scale per 128 columns.  The norm takes h before its rounding: the total's own rounding touches the total only.
// kTeam threads hold a row between its two passes (sum of squares, normalisation), kVecs vectors of 16 columns each, so
// everything is read and written once: HBM-bound.  kTeam <= 32: rows share a warp; kTeam = 0: the whole thread block
// holds one row.  A row whose squares leave fp32 comes out as NaN, and raises VAE_ERR_RANGE with it.
// kKeep, for many rows: the block goes over the rows and keeps gamma and beta in shared memory, laid out so that a warp's
// reads touch each bank once.  Read from global memory for every row, 16 bytes of each 64, they fill the L1 cache's pipe
// (83% busy; 73920 x 1024 bf16 107 us, in pieces of 32 bytes 89, kept 87: 6.1 TB/s; with an fp32 residual 127: 6.5 TB/s).
// A row per thread block: 36000 x 2048 bf16 88 us, 5.8 TB/s; above 12288 columns 4620 x 16384 121, 4.4 (fp32 residual 159,
// 5.2), 2310 x 32768 137, 3.9: one row's barrier holds up its loads, and few blocks fit an SM.
template <typename TX, typename TR, int kTeam, int kVecs, bool kKeep, bool kTiny>
__global__ void __launch_bounds__(kTeam ? kThreads : kRowThreads<kVecs>, (kRmsBlocks<TX, TR, kTeam, kVecs>))
    residual_rms_fp8_kernel(const __grid_constant__ Fp8RmsParams p) {
  constexpr int kT = kTeam ? kTeam : 1;  // (divisor)
  __shared__ float part[2][32];
  extern __shared__ __align__(16) float4 params[];  // kKeep: gamma, beta: [vector][quarter of it][thread of the team]
  const int team = kTeam ? kTeam : static_cast<int>(blockDim.x);
  const int t = kTeam ? threadIdx.x % kT : threadIdx.x;
  const int step = kTeam ? kThreads / kT : 1;  // rows of a block
  const int quads = kVecs * 4 * team;
  if constexpr (kKeep) {
    for (int i = threadIdx.x; i < 2 * quads; i += blockDim.x) {
      const int j = i < quads ? i : i - quads;
      const float* src = i < quads ? p.gamma : p.beta;
      const int col = (j / (4 * team) * team + j % team) * kLane + j / team % 4 * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (src) {
        if (col < p.cols) v.x = __ldg(src + col);
        if (col + 1 < p.cols) v.y = __ldg(src + col + 1);
        if (col + 2 < p.cols) v.z = __ldg(src + col + 2);
        if (col + 3 < p.cols) v.w = __ldg(src + col + 3);
      }
      params[i] = v;
    }
    __syncthreads();
  }
  bool ok = true;
  int turn = 0;
  // (rows of a block that lie behind the last one are counted in 32 bits)
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * step; row0 < p.rows; row0 += static_cast<int64_t>(gridDim.x) * step) {
    const int row = static_cast<int>(row0) + (kTeam ? threadIdx.x / kT : 0);
    F2 h[kVecs][kLane / 2];
    {
      LaneVec<TX> x[kVecs];
#pragma unroll
      for (int k = 0; k < kVecs; ++k)
        load_vec(x[k], static_cast<const TX*>(p.x), p.ld_x, p.rows, p.cols, row, (k * team + t) * kLane, p.ax32);
      if (p.residual) {
        LaneVec<TR> r[kVecs];
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
          load_vec(r[k], static_cast<const TR*>(p.residual), p.ld_residual, p.rows, p.cols, row, (k * team + t) * kLane, p.ar32);
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
    const float2 sp = f2_get(s2);
    float ss = sp.x + sp.y;
#pragma unroll
    for (int d = 1; d < (kTeam ? kTeam : 32); d *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, d);
    if constexpr (kTeam == 0) ss = block_sum(ss, part[turn++ & 1]);
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
        store_vec(static_cast<TR*>(p.total), v, p.ld_total, p.rows, p.cols, row, (k * team + t) * kLane, p.at32);
      }
    }
    float r = inverse_rms(p, ss);
    if constexpr (kTiny) {
      const bool tiny = tiny_mean(p, ss);
      if (__any_sync(0xffffffffu, tiny)) {  // (kTeam 0: in all of the block's warps, or none)
        const float scale = tiny ? kTinyScale : 1.0f;
        s2 = f2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kVecs; ++k)
#pragma unroll
          for (int i = 0; i < kLane / 2; ++i) {
            h[k][i] = f2_mul(h[k][i], f2(scale, scale));
            s2 = f2_fma(h[k][i], h[k][i], s2);
          }
        const float2 sq = f2_get(s2);
        ss = sq.x + sq.y;
#pragma unroll
        for (int d = 1; d < (kTeam ? kTeam : 32); d *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, d);
        if constexpr (kTeam == 0) ss = block_sum(ss, part[turn++ & 1]);
        if (tiny) r = inverse_rms_scaled(p, ss);
      }
    }
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int col = (k * team + t) * kLane;
      if constexpr (kKeep) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 g = params[(k * 4 + j) * team + t], b = params[quads + (k * 4 + j) * team + t];
          h[k][2 * j] = f2_fma(f2_mul(h[k][2 * j], f2(r, r)), f2(g.x, g.y), f2(b.x, b.y));
          h[k][2 * j + 1] = f2_fma(f2_mul(h[k][2 * j + 1], f2(r, r)), f2(g.z, g.w), f2(b.z, b.w));
        }
      } else {
        F2 g[kLane / 2], b[kLane / 2];
        load_params(g, p.gamma, col, p.cols, p.pvec);
#pragma unroll
        for (int i = 0; i < kLane / 2; ++i) b[i] = 0;
        if (p.beta) load_params(b, p.beta, col, p.cols, p.pvec);
#pragma unroll
        for (int i = 0; i < kLane / 2; ++i) h[k][i] = f2_fma(f2_mul(h[k][i], f2(r, r)), g[i], b[i]);
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
  }
  if (!ok) raise_fault(p.fault, FAULT_RANGE, 47);
}

// The same for rows that start anywhere: a warp per row of up to 1024 columns, or (kWide) a thread block per row, each
// warp kBlocks blocks of 128 columns, 4 values of a block per lane.  Bound by issue: 40013 x 333 bf16 with SiLU 28.5 us,
// 9241 x 8191 bf16 162, 3.3 TB/s both; with an fp32 residual 40013 x 333 30.9, 4.7, 9241 x 8191 204, 4.1; 4619 x 16383
// bf16 178, 3.0.
template <typename TX, typename TR, int kBlocks, bool kWide, bool kTiny>
__global__ void __launch_bounds__(kWide ? 512 : kThreads, kWide ? 0 : 4)
    residual_rms_fp8_any_kernel(const __grid_constant__ Fp8RmsParams p) {
  __shared__ float part[kTiny ? 2 : 1][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = kWide ? static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x) * (kThreads / 32) + warp;
  const int first = kWide ? warp : 0, step = kWide ? static_cast<int>(blockDim.x >> 5) : 1;
  if (!kWide && row >= p.rows) return;
  const int have = (p.cols + kFp8Block - 1) / kFp8Block;  // blocks of a row
  float h[kBlocks][4];
  {
    Piece<TX> x[kBlocks];
    Piece<TR> r[kBlocks];
    const TX* px = static_cast<const TX*>(p.x) + row * p.ld_x + lane * 4;
    const TR* pr = static_cast<const TR*>(p.residual) + row * p.ld_residual + lane * 4;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      const int block = first + i * step;
      if (block >= have) break;
      const int n = p.cols - block * kFp8Block - lane * 4;
      x[i].load(px + block * kFp8Block, n);
      if (p.residual) r[i].load(pr + block * kFp8Block, n);
    }
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      if (first + i * step < have) {
        x[i].get(h[i]);
        if (p.residual) {
          float u[4];
          r[i].get(u);
#pragma unroll
          for (int j = 0; j < 4; ++j) h[i][j] += u[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) h[i][j] = 0.f;
      }
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kBlocks; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) ss = fmaf(h[i][j], h[i][j], ss);
#pragma unroll
  for (int d = 1; d < 32; d *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, d);
  if constexpr (kWide) ss = block_sum(ss, part[0]);
  if (p.total) {
    TR* pt = static_cast<TR*>(p.total) + row * p.ld_total + lane * 4;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      const int block = first + i * step;
      if (block >= have) break;
      store4(pt + block * kFp8Block, p.cols - block * kFp8Block - lane * 4, h[i]);
    }
  }
  float r = inverse_rms(p, ss);
  if constexpr (kTiny) {
    if (tiny_mean(p, ss)) {  // (the same for a whole row)
      ss = 0.f;
#pragma unroll
      for (int i = 0; i < kBlocks; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          h[i][j] *= kTinyScale;
          ss = fmaf(h[i][j], h[i][j], ss);
        }
#pragma unroll
      for (int d = 1; d < 32; d *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, d);
      if constexpr (kWide) ss = block_sum(ss, part[1]);
      r = inverse_rms_scaled(p, ss);
    }
  }
  uint8_t* codes = p.codes + static_cast<int64_t>(row) * p.pitch + lane * 4;
  bool ok = true;
#pragma unroll
  for (int i0 = 0; i0 < kBlocks; i0 += 4) {
    if (first + i0 * step >= have) break;
    float m[4], s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = 0.f;
      const int block = first + (i0 + i) * step;
      if (i0 + i >= kBlocks || block >= have) continue;
      const int col = block * kFp8Block + lane * 4;
      float* v = h[i0 + i];
      float4 g = make_float4(0.f, 0.f, 0.f, 0.f), b = g;
      if (p.pvec && col + 4 <= p.cols) {
        g = __ldg(reinterpret_cast<const float4*>(p.gamma + col));
        if (p.beta) b = __ldg(reinterpret_cast<const float4*>(p.beta + col));
      } else {
        if (col < p.cols) g.x = __ldg(p.gamma + col), b.x = p.beta ? __ldg(p.beta + col) : 0.f;
        if (col + 1 < p.cols) g.y = __ldg(p.gamma + col + 1), b.y = p.beta ? __ldg(p.beta + col + 1) : 0.f;
        if (col + 2 < p.cols) g.z = __ldg(p.gamma + col + 2), b.z = p.beta ? __ldg(p.beta + col + 2) : 0.f;
        if (col + 3 < p.cols) g.w = __ldg(p.gamma + col + 3), b.w = p.beta ? __ldg(p.beta + col + 3) : 0.f;
      }
      F2 y[2] = {f2_fma(f2_mul(f2(v[0], v[1]), f2(r, r)), f2(g.x, g.y), f2(b.x, b.y)),
                 f2_fma(f2_mul(f2(v[2], v[3]), f2(r, r)), f2(g.z, g.w), f2(b.z, b.w))};
      if (p.silu) silu<2>(y);
      const float2 y0 = f2_get(y[0]), y1 = f2_get(y[1]);
      v[0] = y0.x; v[1] = y0.y; v[2] = y1.x; v[3] = y1.y;
      m[i] = amax4(v);
    }
    Fp8Scale q[4];
    warp_scales4(m, q, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int block = first + (i0 + i) * step;
      if (i0 + i >= kBlocks || block >= have) continue;
      ok = ok && q[i].finite;
      if (block * kFp8Block + lane * 4 < p.pitch)
        *reinterpret_cast<uint32_t*>(codes + block * kFp8Block) = fp8_codes4(h[i0 + i], q[i]);
      if (lane == 8 * i) p.scales[static_cast<int64_t>(block) * p.rows + row] = s;
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

// What a CUDA call of this library's returned; its error is reported here and does not stay the thread's last one.
vae_status_t status(cudaError_t e) {
  if (e == cudaSuccess) return VAE_OK;
  cudaGetLastError();
  return fail(VAE_ERR_CUDA, "CUDA error: %s", cudaGetErrorString(e));
}
// A launch and its own status: the thread's last error may be an earlier caller's.
template <typename P>
vae_status_t launch(void (*kernel)(P), unsigned grid, int threads, size_t smem, cudaStream_t s, const P& p) {
  void* args[] = {const_cast<P*>(&p)};
  return status(cudaLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(grid), dim3(static_cast<unsigned>(threads)), args, smem, s));
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

// vpr: vectors (or blocks, where rows start anywhere) per row
void fill(Fp8Params& p, const vae_fp8_desc_t* d, const void* values, int vpr) {
  p.rows = static_cast<int>(d->rows);
  p.cols = d->cols;
  p.ld = d->ld;
  p.pitch = (d->cols + 15) / 16 * 16;
  p.row_shift = d->block_rows == 1 ? 0 : 7;
  p.row_blocks = static_cast<int>((d->rows + d->block_rows - 1) / d->block_rows);
  p.vpr = vpr;
  p.vpr_magic = static_cast<uint32_t>(((1ull << 32) + p.vpr - 1) / p.vpr);
  p.vpr_magic64 = ~uint64_t(0) / p.vpr + 1;  // (2^64 / vpr rounded up, unless vpr is 1)
  p.a32 = aligned(values, 32) && (d->ld * size_of(d->dtype)) % 32 == 0;
  p.fault = fault_word();
}

template <typename T>
vae_status_t launch_quantize(const Fp8Params& p, bool vec, bool blocks, unsigned grid, cudaStream_t s) {
  if (blocks) {
    if (vec) return launch(quantize_fp8_block_kernel<T, true>, grid, kThreads, 0, s, p);
    return launch(quantize_fp8_block_kernel<T, false>, grid, kThreads, 0, s, p);
  }
  if (vec) return launch(quantize_fp8_kernel<T>, grid, kThreads, 0, s, p);
  return launch(quantize_fp8_any_kernel<T>, grid, kThreads, 0, s, p);
}
template <typename T>
vae_status_t launch_dequantize(const Fp8Params& p, bool vec, unsigned grid, cudaStream_t s) {
  if (vec) return launch(dequantize_fp8_kernel<T>, grid, kThreads, 0, s, p);
  return launch(dequantize_fp8_any_kernel<T>, grid, kThreads, 0, s, p);
}

// One block per group of rows, or (teams, many rows) blocks that go over the rows and keep the parameters.  Blocks that
// hold one row do not: each row's barrier would hold up the next row's loads (36000 x 2048 bf16 131 us, this way 87).
template <typename TX, typename TR, int kTeam, int kVecs>
vae_status_t launch_rms_team(const Fp8RmsParams& p, int threads, int n_sm, cudaStream_t s) {
  const int step = kTeam ? kThreads / (kTeam ? kTeam : 1) : 1;
  const int64_t groups = (static_cast<int64_t>(p.rows) + step - 1) / step;
  const int64_t many = static_cast<int64_t>(n_sm) * 8;  // blocks: all that fit the SMs, and as many to follow them
  if (p.eps < kTinyMean)
    return launch(residual_rms_fp8_kernel<TX, TR, kTeam, kVecs, false, true>, static_cast<unsigned>(groups), threads, 0, s, p);
  if constexpr (kTeam != 0) {
    if (groups > 2 * many) {
      constexpr size_t kBytes = size_t(2) * kVecs * 4 * kTeam * sizeof(float4);
      return launch(residual_rms_fp8_kernel<TX, TR, kTeam, kVecs, true, false>, static_cast<unsigned>(many), threads, kBytes, s, p);
    }
  }
  return launch(residual_rms_fp8_kernel<TX, TR, kTeam, kVecs, false, false>, static_cast<unsigned>(groups), threads, 0, s, p);
}

// The smallest team whose threads, with two vectors each at most, hold a row (rows of up to 512 columns: one vector each;
// above 12288: four).
template <typename TX, typename TR>
vae_status_t launch_rms(const Fp8RmsParams& p, bool vec, cudaStream_t s) {
  if (vec) {
    int dev = 0, n_sm = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return status(e);
    if (p.cols <= 128) return launch_rms_team<TX, TR, 8, 1>(p, kThreads, n_sm, s);
    if (p.cols <= 256) return launch_rms_team<TX, TR, 16, 1>(p, kThreads, n_sm, s);
    if (p.cols <= 512) return launch_rms_team<TX, TR, 32, 1>(p, kThreads, n_sm, s);
    if (p.cols <= 1024) return launch_rms_team<TX, TR, 32, 2>(p, kThreads, n_sm, s);
    if (p.cols <= kRowThreads<2> * 2 * kLane) return launch_rms_team<TX, TR, 0, 2>(p, (p.cols + 1023) / 1024 * 32, n_sm, s);
    return launch_rms_team<TX, TR, 0, 4>(p, (p.cols + 2047) / 2048 * 32, n_sm, s);
  }
  const int blocks = (p.cols + kFp8Block - 1) / kFp8Block;
  if (blocks <= 8) {
    const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(p.rows) + kThreads / 32 - 1) / (kThreads / 32));
    if (p.eps < kTinyMean) return launch(residual_rms_fp8_any_kernel<TX, TR, 8, false, true>, grid, kThreads, 0, s, p);
    if (blocks <= 1) return launch(residual_rms_fp8_any_kernel<TX, TR, 1, false, false>, grid, kThreads, 0, s, p);
    if (blocks <= 2) return launch(residual_rms_fp8_any_kernel<TX, TR, 2, false, false>, grid, kThreads, 0, s, p);
    if (blocks <= 4) return launch(residual_rms_fp8_any_kernel<TX, TR, 4, false, false>, grid, kThreads, 0, s, p);
    return launch(residual_rms_fp8_any_kernel<TX, TR, 8, false, false>, grid, kThreads, 0, s, p);
  }
  const unsigned rows = static_cast<unsigned>(p.rows);
  if (p.eps < kTinyMean) return launch(residual_rms_fp8_any_kernel<TX, TR, 16, true, true>, rows, (blocks + 15) / 16 * 32, 0, s, p);
  // (20001 x 3001: 4 blocks a warp 120 us, 8 132; 9241 x 8191: 189, 162)
  if (blocks <= 32) return launch(residual_rms_fp8_any_kernel<TX, TR, 4, true, false>, rows, (blocks + 3) / 4 * 32, 0, s, p);
  if (blocks <= 128) return launch(residual_rms_fp8_any_kernel<TX, TR, 8, true, false>, rows, (blocks + 7) / 8 * 32, 0, s, p);
  return launch(residual_rms_fp8_any_kernel<TX, TR, 16, true, false>, rows, (blocks + 15) / 16 * 32, 0, s, p);
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
  const bool vec = aligned(x, 16) && (d->ld * esz) % 16 == 0;
  const bool blocks = d->block_rows != 1;
  const int nc = (d->cols + kFp8Block - 1) / kFp8Block;
  fill(p, d, x, vec && !blocks ? nc * kFp8Team : nc);
  p.x = x;
  p.y = codes;
  p.scales = scales;
  const int64_t per_block = vec ? kThreads * kVptIn : kThreads / 32 * kUnits;
  const int64_t grid = blocks ? static_cast<int64_t>(p.row_blocks) * nc : (d->rows * p.vpr + per_block - 1) / per_block;
  if (grid > 0x7fffffffLL) return fail(VAE_ERR_UNSUPPORTED, "too many values for one call");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d->dtype == VAE_FP32) return launch_quantize<float>(p, vec, blocks, static_cast<unsigned>(grid), s);
  return launch_quantize<__nv_bfloat16>(p, vec, blocks, static_cast<unsigned>(grid), s);
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
  const bool vec = aligned(y, 16) && (d->ld * esz) % 16 == 0;
  fill(p, d, y, vec ? (d->cols + kLane - 1) / kLane : (d->cols + kFp8Block - 1) / kFp8Block);
  p.x = codes;
  p.y = y;
  p.scales = const_cast<float*>(scales);
  const int64_t per_block = vec ? kThreads * kVptOut : kThreads / 32 * kUnits;
  const int64_t grid = (d->rows * p.vpr + per_block - 1) / per_block;
  if (grid > 0x7fffffffLL) return fail(VAE_ERR_UNSUPPORTED, "too many values for one call");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d->dtype == VAE_FP32) return launch_dequantize<float>(p, vec, static_cast<unsigned>(grid), s);
  return launch_dequantize<__nv_bfloat16>(p, vec, static_cast<unsigned>(grid), s);
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
  return status(launch_gemm_fp8(a, static_cast<cudaStream_t>(stream)));
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
  p.pvec = aligned(gamma, 32) && aligned(beta, 32);
  p.fault = fault_word();
  const bool vec = aligned(x, 16) && (d->ld_x * ex) % 16 == 0 &&
                   (!residual || (aligned(residual, 16) && (d->ld_residual * er) % 16 == 0)) &&
                   (!total || (aligned(total, 16) && (d->ld_total * er) % 16 == 0));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  using bf16 = __nv_bfloat16;
  const bool xf = d->dtype == VAE_FP32, rf = d->residual_dtype == VAE_FP32;
  if (xf && rf) return launch_rms<float, float>(p, vec, s);
  if (xf) return launch_rms<float, bf16>(p, vec, s);
  if (rf) return launch_rms<bf16, float>(p, vec, s);
  return launch_rms<bf16, bf16>(p, vec, s);
}
