// What the elementwise kernels of the 4-bit and 8-bit operands share: fp32 pairs, 16 values of a row per lane, SiLU and
// correctly rounded quotients of them.
#pragma once

#include "common.cuh"

namespace vae {

// max(|a|, |b|, |c|), NaN when any is NaN
VAE_DEV float max_abs_or_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Two fp32 values in one 64-bit register, and arithmetic on both at once (one issue slot; each rounds as usual).
using F2 = uint64_t;
VAE_DEV F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
VAE_DEV float2 f2_get(F2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
VAE_DEV F2 f2_mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
VAE_DEV F2 f2_add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
VAE_DEV F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// What a lane holds of a row: 16 values (32 bytes of bf16, 64 of fp32), taken as 8 pairs.  Half a MXFP4 block, a whole
// NVFP4 block, an eighth of an 8-bit block: the work per block (its scale, its shuffles, its addresses) is shared by as
// many values as fit registers.
constexpr int kLane = 16;
template <typename T> struct LaneVec {
  static constexpr int kW = kLane * static_cast<int>(sizeof(T)) / 4;
  uint32_t w[kW];
  VAE_DEV void zero() {
#pragma unroll
    for (int i = 0; i < kW; ++i) w[i] = 0u;
  }
  // a32: the address is 32-byte aligned (32-byte loads), else 16-byte aligned
  VAE_DEV void load(const T* p, bool a32) {
    const uint4* q = reinterpret_cast<const uint4*>(p);
    if (a32) {
#pragma unroll
      for (int i = 0; i < kW; i += 8)
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]), "=r"(w[i + 4]), "=r"(w[i + 5]),
                       "=r"(w[i + 6]), "=r"(w[i + 7])
                     : "l"(q + i / 4));
    } else {
#pragma unroll
      for (int i = 0; i < kW; i += 4) {
        const uint4 a = q[i / 4];
        w[i] = a.x; w[i + 1] = a.y; w[i + 2] = a.z; w[i + 3] = a.w;
      }
    }
  }
  VAE_DEV void get(F2* v) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 2) v[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
      else v[i] = f2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    }
  }
};

// A lane's 16 values to memory as T; a32 as above.
VAE_DEV void store_lane(float* p, const float* v, bool a32) {
  if (a32) {
#pragma unroll
    for (int i = 0; i < 16; i += 8)
      asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + i), "f"(v[i]), "f"(v[i + 1]),
                   "f"(v[i + 2]), "f"(v[i + 3]), "f"(v[i + 4]), "f"(v[i + 5]), "f"(v[i + 6]), "f"(v[i + 7])
                   : "memory");
  } else {
    store8(p, v);
    store8(p + 8, v + 8);
  }
}
VAE_DEV void store_lane(__nv_bfloat16* p, const float* v, bool a32) {
  if (a32) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    store8(p, v);
    store8(p + 8, v + 8);
  }
}

// Element e = 32 i + lane of the 512 that a warp's vectors hold lies in the vector of lane e / 16: its row and column, so
// that a warp reads or writes rows that start anywhere 32 adjacent elements at a time.
VAE_DEV void element_of(int i, int lane, int row, int col, int& erow, int& ecol) {
  const int e = i * 32 + lane;
  erow = __shfl_sync(0xffffffffu, row, e / kLane);
  ecol = __shfl_sync(0xffffffffu, col, e / kLane) + e % kLane;
}

// SiLU z / (1 + exp(-z)) of a lane's values: two special function operations per value.  Off by a few units in the last
// place, and for negative z by |z| 2^-24 of itself more (the rounding of z log2 e, in the exponent); below about -87.3,
// where it is smaller than 2^-119, it comes out as zero.
// (One reciprocal for two values, 1 / a = b / (a b), with a branch for products that leave fp32, gains nothing: group norm
// + SiLU into MXFP4 on 21 x 88 x 160 x 512 with its product 239 us, this way 236.)
template <int kPairs = kLane / 2>
VAE_DEV void silu(F2* z) {
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    float2 e = f2_get(f2_mul(z[i], f2(-1.4426950408889634f, -1.4426950408889634f)));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.x));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.y));
    float2 a = f2_get(f2_add(f2(e.x, e.y), f2(1.0f, 1.0f)));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a.x));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a.y));
    z[i] = f2_mul(z[i], f2(a.x, a.y));
  }
}

// x / d rounded to fp32, from nd = -d and r = 1 / d correctly rounded: q0 = x r, then q0 + (x - q0 d) r with fused
// multiply-adds is the correctly rounded quotient (P. W. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", IBM J. Res. Dev. 34, 1990).  With d = r = 0 it gives zeros; an x of -0 gives +0.
VAE_DEV float div_by(float x, float nd, float r) {
  const float q0 = x * r;
  return fmaf(fmaf(q0, nd, x), r, q0);
}
VAE_DEV F2 div_by(F2 x, F2 nd, F2 r) {
  const F2 q0 = f2_mul(x, r);
  return f2_fma(f2_fma(q0, nd, x), r, q0);
}

}  // namespace vae
