// Microscaled 4-bit operands: element conversions, block scales and the layouts the kernels share.
//
// Elements are e2m1 (1 sign, 2 exponent, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two to a byte, the
// element of the lower column in the low nibble.  MXFP4 gives each 32 columns of a row one power-of-two
// scale (8-bit exponent, bias 127); NVFP4 gives each 16 columns one e4m3 scale, times one fp32 tensor scale.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace vae {

// 4-block scale groups of a row of `cols` columns
inline int fp4_groups(int format, int cols) {
  const int block = format == VAE_MXFP4 ? 32 : 16;
  return ((cols + block - 1) / block + 3) / 4;
}

// Block scales lie in tiles of 128 rows x 4 blocks, 512 bytes each, the 4-block groups of one row tile
// next to each other: the form tcgen05.cp (32 lanes x 16 bytes) brings into tensor memory, where lane
// r % 32 of column r / 32 of a tile holds row r's 4 bytes.
VAE_DEV int64_t fp4_scale_offset(int64_t row, int block, int groups) {
  return ((row >> 7) * groups + (block >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 + (block & 3);
}

// max(a, |x|) that is NaN when either is NaN
VAE_DEV float max_abs_or_nan(float a, float x) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(x)));
  return r;
}

// 8 values -> 8 e2m1 codes (round to nearest, ties to the even code, beyond 6 saturated), v[0] lowest.
VAE_DEV uint32_t e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// 8 e2m1 codes -> values (exact in half precision)
VAE_DEV void e2m1x8_values(uint32_t codes, float* v) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

// The value of a scale byte (without the tensor scale).
template <int kFmt>
VAE_DEV float fp4_scale_value(uint32_t byte) {
  if constexpr (kFmt == VAE_MXFP4) {
    if (byte == 255u) return __int_as_float(0x7fffffff);
    return __uint_as_float(byte ? byte << 23 : 0x00400000u);  // 2^(byte - 127); 2^-127 is subnormal
  } else {
    __nv_fp8_e4m3 s;
    s.__x = static_cast<__nv_fp8_storage_t>(byte);
    return static_cast<float>(s);
  }
}

// SiLU z / (1 + exp(-z)) of 8 values, to a few units in the last place.  exp is one MUFU operation (ex2) per value and
// the reciprocal one per two, 1 / a = b / (a b): the special function units are what bounds this pass otherwise.
// Where a product a b leaves fp32 (both z below about -43) the reciprocals are taken one by one.
VAE_DEV void silu8(float* z) {
  float a[8], r[4];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z[i] * -1.4426950408889634f));
    a[i] = 1.0f + e;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r[i]) : "f"(a[2 * i] * a[2 * i + 1]));
  if (fminf(fminf(r[0], r[1]), fminf(r[2], r[3])) > 0.f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[2 * i] *= r[i] * a[2 * i + 1];
      z[2 * i + 1] *= r[i] * a[2 * i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(a[i]));
      z[i] *= s;
    }
  }
}

// Lanes that share a block, each holding 8 consecutive columns of it.
template <int kFmt> constexpr int kFp4Team = kFmt == VAE_MXFP4 ? 4 : 2;
template <int kFmt> constexpr int kFp4Block = kFmt == VAE_MXFP4 ? 32 : 16;

// What a kernel needs of a format's tensor scale t: t, 6 t and 1 / (6 t), each rounded to fp32, and the block maximum
// from which on every scale is clipped (6 t 512; it keeps the quotients finite).
struct Fp4Scale {
  float t, t6, r6, top;
};
inline Fp4Scale fp4_scale(float t) { return Fp4Scale{t, 6.0f * t, 1.0f / (6.0f * t), 6.0f * t * 512.0f}; }

// x / d rounded to fp32, from r = 1 / d correctly rounded: q0 = x r, then q0 - (q0 d - x) r with fused multiply-adds
// is the correctly rounded quotient (P. W. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", IBM J. Res. Dev. 34, 1990).  Written this way round it keeps the sign of a zero x, and with
// d = r = 0 it gives zeros.
VAE_DEV float div_by(float x, float d, float r) {
  const float q0 = x * r;
  return fmaf(-fmaf(q0, d, -x), r, q0);
}

// Quantise 8 columns of a block: v is this lane's 8 values, the block's other columns lie in the other
// lanes of its team (all 32 lanes of the warp call this together).  Returns the codes; `byte` gets the
// block's scale byte (the same in every lane of the team) and `ok` whether the format could hold the block.
//
// MXFP4: the scale is the power of two 2^e with max|x| in [3.5, 7) 2^e.  Below 7 the largest value rounds
// to at most 6 with an error of half the last step, so nothing is clipped; the rule is one addition to
// the bits of max|x| (mantissas from 1.75 on carry into the exponent).  On normal values the relative
// rms error is 0.112, against 0.115 with the exponent of max|x| alone, which clips (6, 8), and
// 0.115 with the next power of two above max|x| / 6.  x / 2^e is exact.
// NVFP4: the scale is max|x| / (6 t) rounded to the nearest e4m3 value s, t the tensor scale, and the codes
// round x / (s t), s t in fp32.  Both quotients are correctly rounded to fp32; with t a power of two such a quotient lies
// on the same side of every e4m3 or e2m1 rounding border as the true one.
// A NaN or an infinity in the block makes its scale NaN (and the codes 0): it reads back, and multiplies,
// as NaN.  An NVFP4 block whose scale would pass 448 (rounding from 464) is clipped.  Both clear `ok`.
template <int kFmt>
VAE_DEV uint32_t fp4_quantize8(const float* v, const Fp4Scale& ts, uint32_t& byte, bool& ok) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max_abs_or_nan(amax, v[i]);
#pragma unroll
  for (int off = kFp4Team<kFmt> >> 1; off > 0; off >>= 1)
    amax = max_abs_or_nan(amax, __shfl_xor_sync(0xffffffffu, amax, off));
  const bool finite = amax < __int_as_float(0x7f800000);
  float q[8];
  if constexpr (kFmt == VAE_MXFP4) {
    const int e = max(static_cast<int>((__float_as_uint(amax) + 0x200000u) >> 23) - 2, 0);
    byte = finite ? static_cast<uint32_t>(e) : 255u;
    const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);  // 2^(127 - e), e <= 253
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = v[i] * inv;
    ok = finite;
  } else {
    const float s6 = div_by(fminf(amax, ts.top), ts.t6, ts.r6);
    const uint32_t s8 = __nv_cvt_float_to_fp8(s6, __NV_SATFINITE, __NV_E4M3);
    byte = finite ? s8 : 127u;
    ok = finite && s6 <= 464.f;
    const float st = fp4_scale_value<kFmt>(s8) * ts.t;
    const float r = st > 0.f ? __frcp_rn(st) : 0.f;  // (s = 0: max|x| below half the smallest scale, the block is zeros)
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = div_by(v[i], st, r);
    if (!ok) {  // clipped: the quotients may have overflowed on the way
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = div_by(fminf(fmaxf(v[i], -8.f * st), 8.f * st), st, r);
    }
  }
  const uint32_t codes = e2m1x8(q);
  return finite ? codes : 0u;
}

}  // namespace vae
