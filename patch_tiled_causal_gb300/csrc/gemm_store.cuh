// How the products of low-precision operands store their results: a warp's 32 rows x 128 bytes through a swizzled
// shared-memory buffer, by TMA where D allows it, row by row elsewhere.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace vae {

constexpr uint32_t kStoreBuf = 32u * 128u;  // bytes of one store buffer (32 rows x 128 bytes)

// P: the product's parameters with M, N (sizes of D), y, ldd (D and its row stride), vec (rows of D start on 16-byte
// boundaries) and whole16 (they are whole 16-byte chunks long).
// Columns [c0, c0 + kCols) of this warp's accumulator rows -> its store buffer -> D.  v: alpha * acc + bias.
template <typename TO, typename P>
VAE_DEV void store_slab(const P& p, const CUtensorMap* tmD, uint8_t* buf, const float* v, int row0, int n0,
                        int lane) {
  constexpr int kCols = 128 / static_cast<int>(sizeof(TO));
  // 16-byte chunk c of row r sits at chunk c ^ (r & 7): the 128-byte swizzle of the store's tensor map, and free of
  // bank conflicts for one row per lane
  uint8_t* dst = buf + lane * 128;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint4 u;
    if constexpr (sizeof(TO) == 2) {
      __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[8 * c + 2 * i], v[8 * c + 2 * i + 1]);
    } else {
      u = make_uint4(__float_as_uint(v[4 * c]), __float_as_uint(v[4 * c + 1]), __float_as_uint(v[4 * c + 2]),
                     __float_as_uint(v[4 * c + 3]));
    }
    *reinterpret_cast<uint4*>(dst + ((c ^ (lane & 7)) << 4)) = u;
  }
  // (a store ends at whole 16-byte chunks of a row: past D's last column where N does not fill the chunk)
  if (p.vec && (p.whole16 || n0 + kCols <= p.N)) {
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) {
      if (row0 < p.M && n0 < p.N) tma_store_2d(tmD, smem_u32(buf), n0, row0);
      bulk_commit();
    }
  } else {
    __syncwarp();
    // 8 rows at a time, all shared-memory reads before the first store
    const int rows = min(32, p.M - row0), cols = min(kCols, p.N - n0);
    for (int r0 = 0; r0 < rows; r0 += 8) {
      TO t[8][kCols / 32];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < kCols / 32; ++j)
          t[i][j] = *reinterpret_cast<const TO*>(
              buf + (r0 + i) * 128 + (((lane + 32 * j) * static_cast<int>(sizeof(TO))) ^ (i << 4)));
      TO* out = static_cast<TO*>(p.y) + static_cast<int64_t>(row0 + r0) * p.ldd + n0 + lane;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int j = 0; j < kCols / 32; ++j)
          if (r0 + i < rows && lane + 32 * j < cols) out[32 * j] = t[i][j];
        out += p.ldd;
      }
    }
    __syncwarp();
    if (lane == 0) bulk_commit();  // (an empty group: one for each slab, whichever way it goes)
  }
}

}  // namespace vae
