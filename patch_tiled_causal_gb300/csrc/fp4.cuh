// Microscaled 4-bit operands: element conversions, block scales and the layouts the kernels share.
//
// Elements are e2m1 (1 sign, 2 exponent, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two to a byte, the
// element of the lower column in the low nibble.  MXFP4 gives each 32 columns of a row one power-of-two
// scale (8-bit exponent, bias 127); NVFP4 gives each 16 columns one e4m3 scale, times one fp32 tensor scale.
#pragma once

#include <cuda_fp16.h>

#include "internal.h"
#include "lane.cuh"

namespace vae {

// 4-block scale groups of a row of `cols` columns
inline int fp4_groups(int format, int cols) {
  const int block = format == VAE_MXFP4 ? 32 : 16;
  return ((cols + block - 1) / block + 3) / 4;
}

// Block scales lie in tiles of 128 rows x 4 blocks, 512 bytes each, the 4-block groups of one row tile
// next to each other: the form tcgen05.cp (32 lanes x 16 bytes) brings into tensor memory, where lane
// r % 32 of column r / 32 of a tile holds row r's 4 bytes.
// (An operand has fewer than 2^31 rows and at most 2^40 values, so its scale tiles are counted in 32 bits.)
VAE_DEV uint64_t fp4_scale_offset(int row, int block, int groups) {
  const uint32_t tile = static_cast<uint32_t>(row >> 7) * static_cast<uint32_t>(groups) + static_cast<uint32_t>(block >> 2);
  return static_cast<uint64_t>(tile) * 512u + static_cast<uint32_t>((row & 31) * 16 + ((row >> 5) & 3) * 4 + (block & 3));
}

// 4 pairs of values -> 8 e2m1 codes (round to nearest, ties to the even code, beyond 6 saturated), v[0] lowest.
VAE_DEV uint32_t e2m1x8(const F2* v) {
  const float2 a = f2_get(v[0]), b = f2_get(v[1]), c = f2_get(v[2]), d = f2_get(v[3]);
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
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

template <int kFmt> constexpr int kFp4Block = kFmt == VAE_MXFP4 ? 32 : 16;

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

// Lanes that share a block, each holding kLane consecutive columns of it.
template <int kFmt> constexpr int kFp4Team = kFp4Block<kFmt> / kLane;

// What a kernel needs of a format's tensor scale t: t, 6 t and 1 / (6 t), each rounded to fp32, and the block maximum
// from which on every scale is clipped (6 t 512; it keeps the quotients finite).
struct Fp4Scale {
  float t, t6, r6, top;
};
inline Fp4Scale fp4_scale(float t) { return Fp4Scale{t, 6.0f * t, 1.0f / (6.0f * t), 6.0f * t * 512.0f}; }

// Quantise kLane columns of a block: v is this lane's values, the block's other columns lie in the other
// lane of its team (all 32 lanes of the warp call this together).  codes gets the 2 words, `byte` the block's
// scale byte (the same in every lane of the team) and `ok` whether the format could hold the block.
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
VAE_DEV void fp4_quantize(const F2* v, const Fp4Scale& ts, uint2& codes, uint32_t& byte, bool& ok) {
  // 16 values in three levels of three
  float x[16], m[5];
#pragma unroll
  for (int i = 0; i < kLane / 2; ++i) {
    const float2 t = f2_get(v[i]);
    x[2 * i] = t.x;
    x[2 * i + 1] = t.y;
  }
#pragma unroll
  for (int i = 0; i < 5; ++i) m[i] = max_abs_or_nan(x[3 * i], x[3 * i + 1], x[3 * i + 2]);
  float amax = max_abs_or_nan(max_abs_or_nan(m[0], m[1], m[2]), max_abs_or_nan(m[3], m[4], x[15]), 0.f);
  if constexpr (kFp4Team<kFmt> == 2) amax = max_abs_or_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1), 0.f);
  const bool finite = amax < __int_as_float(0x7f800000);
  F2 q[kLane / 2];
  if constexpr (kFmt == VAE_MXFP4) {
    const int e = max(static_cast<int>((__float_as_uint(amax) + 0x200000u) >> 23) - 2, 0);
    byte = finite ? static_cast<uint32_t>(e) : 255u;
    const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);  // 2^(127 - e), e <= 253
#pragma unroll
    for (int i = 0; i < kLane / 2; ++i) q[i] = f2_mul(v[i], f2(inv, inv));
    ok = finite;
  } else {
    const float s6 = div_by(fminf(amax, ts.top), -ts.t6, ts.r6);
    const uint32_t s8 = __nv_cvt_float_to_fp8(s6, __NV_SATFINITE, __NV_E4M3);
    byte = finite ? s8 : 127u;
    ok = finite && s6 <= 464.f;
    const float st = fp4_scale_value<kFmt>(s8) * ts.t;
    const float r = st > 0.f ? __frcp_rn(st) : 0.f;  // (s = 0: max|x| below half the smallest scale, the block is zeros)
    const F2 nst2 = f2(-st, -st), r2 = f2(r, r);
    if (ok) {
#pragma unroll
      for (int i = 0; i < kLane / 2; ++i) q[i] = div_by(v[i], nst2, r2);
    } else {  // clipped: the quotients may overflow on the way
#pragma unroll
      for (int i = 0; i < kLane / 2; ++i) {
        const float2 x = f2_get(v[i]);
        q[i] = div_by(f2(fminf(fmaxf(x.x, -8.f * st), 8.f * st), fminf(fmaxf(x.y, -8.f * st), 8.f * st)), nst2, r2);
      }
    }
  }
  codes = finite ? make_uint2(e2m1x8(q), e2m1x8(q + 4)) : make_uint2(0u, 0u);
}

// The scale bytes of 4 neighbouring blocks as one word, in every lane of their 4 teams (whole warp).
template <int kTeam>
VAE_DEV uint32_t fp4_scale_word(uint32_t byte, int lane) {
  uint32_t word = byte << (8 * ((lane / kTeam) & 3));
  word |= __shfl_xor_sync(0xffffffffu, word, kTeam);
  return word | __shfl_xor_sync(0xffffffffu, word, 2 * kTeam);
}

}  // namespace vae
