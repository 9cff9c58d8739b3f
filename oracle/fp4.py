"""Microscaled 4-bit operands in float64: quantisation, reading back, packing, and the product.

TensorRT-LLM PR #16066 "ParallelVAE_TrtllmWan for native Wan VAE" (reviewer comment) names 4-bit
quantisation fused into the norm and SiLU; the formats are MXFP4 ("mx": e2m1 elements, blocks of 32, a
power-of-two scale) and NVFP4 ("nv": e2m1 elements, blocks of 16, an e4m3 scale, one fp32 tensor scale).
Every function is written from the formats' definitions by table look-up; nothing is shared with the GPU path.
"""
from __future__ import annotations

from typing import Tuple

import numpy as np

BLOCK = {"mx": 32, "nv": 16}

# the magnitudes of the 8 positive codes
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])

# the 127 finite non-negative e4m3 values by byte (bias 7, 3 mantissa bits, subnormals below 2^-6); byte 127 is NaN
E4M3 = np.array([(b & 7) * 2.0 ** -9 if b < 8 else (1 + (b & 7) / 8) * 2.0 ** ((b >> 3) - 7) for b in range(127)])


def nearest_even(a: np.ndarray, table: np.ndarray) -> np.ndarray:
    """Index of the entry of the ascending table nearest to each a >= 0 (ties to the even index; beyond the
    last entry, the last)."""
    hi = np.clip(np.searchsorted(table, a), 1, len(table) - 1)
    lo = hi - 1
    mid = (table[lo] + table[hi]) / 2
    up = (a > mid) | ((a == mid) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def quantize(x: np.ndarray, fmt: str, tensor_scale: float = 1.0) -> Tuple[np.ndarray, np.ndarray]:
    """x [rows, cols] -> (codes [rows, cols] 0..15, scale bytes [rows, blocks]).

    mx: scale 2^e, e the exponent with max|x| in [3.5, 7) 2^e (at least -127); nv: the e4m3 value nearest
    max|x| / (6 t).  Quotients of nv are fp32 numbers, as are 6 t and s t.  A block with a NaN or an infinity has
    a NaN scale and codes 0."""
    rows, cols = x.shape
    blk = BLOCK[fmt]
    nb = -(-cols // blk)
    pad = np.zeros((rows, nb * blk))
    pad[:, :cols] = x
    v = pad.reshape(rows, nb, blk)
    bad = ~np.isfinite(v).all(axis=2)
    v = np.where(bad[..., None], 0.0, v)
    sign = np.where(bad[..., None], False, np.signbit(pad.reshape(rows, nb, blk)))
    amax = np.abs(v).max(axis=2)
    if fmt == "mx":
        mant, ex = np.frexp(amax)  # amax = mant * 2^ex, mant in [0.5, 1)
        e = np.where(amax > 0, ex - 3 + (mant >= 0.875), -127)
        e = np.maximum(e, -127)
        byte = np.where(bad, 255, e + 127)
        q = v / np.exp2(e.astype(np.float64))[..., None]
    else:
        t6 = float(np.float32(6.0) * np.float32(tensor_scale))
        byte = nearest_even((amax / t6).astype(np.float32).astype(np.float64), E4M3)
        st = (E4M3[byte] * float(np.float32(tensor_scale))).astype(np.float32).astype(np.float64)
        q = np.where(st[..., None] > 0, v / np.where(st > 0, st, 1.0)[..., None], 0.0)
        q = q.astype(np.float32).astype(np.float64)
        byte = np.where(bad, 127, byte)
    codes = nearest_even(np.abs(q), E2M1) + 8 * sign
    return codes.reshape(rows, -1)[:, :cols].astype(np.uint8), byte.astype(np.uint8)


def scale_values(byte: np.ndarray, fmt: str) -> np.ndarray:
    if fmt == "mx":
        return np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127))
    return np.append(E4M3, np.nan)[byte & 127]


def values(codes: np.ndarray, byte: np.ndarray, fmt: str, tensor_scale: float = 1.0) -> np.ndarray:
    """code * scale * tensor_scale of every element [rows, cols]."""
    mag = E2M1[codes & 7]
    v = np.where(codes >= 8, -mag, mag)
    return v * np.repeat(scale_values(byte, fmt), BLOCK[fmt], axis=1)[:, :codes.shape[1]] * float(np.float32(tensor_scale))


def pack_codes(codes: np.ndarray) -> np.ndarray:
    """[rows, cols] codes -> [rows, ceil(cols / 32) * 16] bytes, the lower column in the low nibble."""
    rows, cols = codes.shape
    wide = np.zeros((rows, -(-cols // 32) * 32), dtype=np.uint8)
    wide[:, :cols] = codes
    return wide[:, 0::2] | (wide[:, 1::2] << 4)


def pack_scales(byte: np.ndarray) -> np.ndarray:
    """[rows, blocks] scale bytes -> flat tiles of 128 rows x 4 blocks, byte by byte."""
    rows, nb = byte.shape
    ng = -(-nb // 4)
    out = np.zeros(-(-rows // 128) * ng * 512, dtype=np.uint8)
    for r in range(rows):
        for b in range(nb):
            out[((r // 128) * ng + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] = byte[r, b]
    return out


def gemm(a: np.ndarray, b: np.ndarray, alpha: float = 1.0, bias=None) -> np.ndarray:
    """alpha * a b^T + bias of dequantised operands a [M, K], b [N, K]."""
    d = alpha * (a @ b.T)
    return d if bias is None else d + bias.astype(np.float64)
