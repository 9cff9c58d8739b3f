// 8-bit operands with block scales: e4m3 codes (1 sign, 4 exponent, 3 mantissa bits, largest finite value 448), and one
// fp32 scale for 128 columns of a row (activations) or for 128 columns of 128 rows (weights).
#pragma once

#include <cuda_fp16.h>

#include "lane.cuh"

namespace vae {

constexpr int kFp8Block = 128;
constexpr int kFp8Team = kFp8Block / kLane;  // lanes that share a row's part of a block, kLane columns each

// What quantising a block takes, from its largest magnitude: the scale s, and x k -> x / s as div_by(x k, nsk, r) with
// nsk = -(s k), r = 1 / (s k).
//
// s is the fp32 quotient max|x| / 448, at least 2^-126 (so that it is a normal number and keeps its digits: a block of
// tiny values loses low bits to e4m3's own subnormals instead of being clipped), and the codes round the fp32 quotients
// x / s, both correctly rounded; the largest value becomes 448 to within one rounding, so nothing is clipped.
// Below max|x| = 2^-60 everything is multiplied by k = 2^64 first (exact), as the remainders of the quotients could
// leave fp32's range there.  The e4m3 rounding of such a quotient equals that of the true one, but where the true one
// lies within half an fp32 unit of a border.
// A NaN or an infinity in the block makes s NaN and the codes 0: it reads back, and multiplies, as NaN; finite says so.
struct Fp8Scale {
  float s, nsk, r, k;
  bool finite;
};
VAE_DEV Fp8Scale fp8_scale(float amax) {
  Fp8Scale q;
  q.finite = amax < __int_as_float(0x7f800000);
  const bool tiny = amax < 0x1p-60f;
  q.k = tiny ? 0x1p64f : 1.0f;
  const float sk = fmaxf(div_by(amax * q.k, -448.0f, 1.0f / 448.0f), tiny ? 0x1p-62f : 0x1p-126f);
  q.s = q.finite ? (tiny ? sk * 0x1p-64f : sk) : __int_as_float(0x7fffffff);
  q.nsk = -sk;
  q.r = __frcp_rn(sk);
  return q;
}

// max|x| of a lane's values, NaN when any is NaN
VAE_DEV float lane_amax(const F2* v) {
  float x[kLane], m[5];
#pragma unroll
  for (int i = 0; i < kLane / 2; ++i) {
    const float2 t = f2_get(v[i]);
    x[2 * i] = t.x;
    x[2 * i + 1] = t.y;
  }
#pragma unroll
  for (int i = 0; i < 5; ++i) m[i] = max_abs_or_nan(x[3 * i], x[3 * i + 1], x[3 * i + 2]);
  return max_abs_or_nan(max_abs_or_nan(m[0], m[1], m[2]), max_abs_or_nan(m[3], m[4], x[15]), 0.f);
}
// The same over the lanes of a team (whole warp).
VAE_DEV float team_amax(float m) {
#pragma unroll
  for (int d = 1; d < kFp8Team; d *= 2) m = max_abs_or_nan(m, __shfl_xor_sync(0xffffffffu, m, d), 0.f);
  return m;
}

// 2 pairs of values -> 4 e4m3 codes (round to nearest, ties to even), v[0] lowest.
VAE_DEV uint32_t e4m3x4(F2 v0, F2 v1) {
  const float2 a = f2_get(v0), b = f2_get(v1);
  uint32_t r;
  asm("{\n\t.reg .b16 h0, h1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h0, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h1, %4, %3;\n\t"
      "mov.b32 %0, {h0, h1};\n\t}"
      : "=r"(r)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
// A lane's 16 codes.
VAE_DEV uint4 fp8_codes(const F2* v, const Fp8Scale& q) {
  if (!q.finite) return make_uint4(0u, 0u, 0u, 0u);
  F2 t[kLane / 2];
  const F2 nsk = f2(q.nsk, q.nsk), r = f2(q.r, q.r);
  if (q.k == 1.0f) {
#pragma unroll
    for (int i = 0; i < kLane / 2; ++i) t[i] = div_by(v[i], nsk, r);
  } else {
    const F2 k = f2(q.k, q.k);
#pragma unroll
    for (int i = 0; i < kLane / 2; ++i) t[i] = div_by(f2_mul(v[i], k), nsk, r);
  }
  return make_uint4(e4m3x4(t[0], t[1]), e4m3x4(t[2], t[3]), e4m3x4(t[4], t[5]), e4m3x4(t[6], t[7]));
}

// 4 e4m3 codes -> values (exact in half precision)
VAE_DEV void e4m3x4_values(uint32_t codes, float* v) {
  uint32_t h[2];
  asm("{\n\t.reg .b16 h0, h1;\n\t"
      "mov.b32 {h0, h1}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, h0;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h1;\n\t}"
      : "=r"(h[0]), "=r"(h[1])
      : "r"(codes));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

}  // namespace vae
