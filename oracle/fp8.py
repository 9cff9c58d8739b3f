"""8-bit operands with a scale for each block of 128, in float64: quantisation, reading back, the product, and the RMS
norm of a residual sum.

TensorRT-LLM PR #16066 "ParallelVAE_TrtllmWan for native Wan VAE" (reviewer comment) names low-precision quantisation fused
into the norm; the format is e4m3 with one fp32 scale per 128 columns of 1 or 128 rows.  Every function is written from
the definitions by table look-up; nothing is shared with the GPU path.
"""
from __future__ import annotations

from typing import Optional, Tuple

import numpy as np

from .fp4 import E4M3, nearest_even

BLOCK = 128


def _per_block(x: np.ndarray, block_rows: int) -> np.ndarray:
    """[rows, cols] -> [row blocks, block_rows, column blocks, 128], zeros behind the end."""
    rows, cols = x.shape
    nr, nc = -(-rows // block_rows), -(-cols // BLOCK)
    pad = np.zeros((nr * block_rows, nc * BLOCK))
    pad[:rows, :cols] = x
    return pad.reshape(nr, block_rows, nc, BLOCK)


def quantize(x: np.ndarray, block_rows: int) -> Tuple[np.ndarray, np.ndarray]:
    """x [rows, cols] -> (e4m3 bytes [rows, cols], fp32 scales [column blocks, row blocks]).

    The scale is the fp32 quotient max|x| / 448, at least 2^-126; the codes round the fp32 quotients x / scale.  A block
    with a NaN or an infinity has a NaN scale and codes 0."""
    rows, cols = x.shape
    v = _per_block(x, block_rows)
    bad = ~np.isfinite(v).all(axis=(1, 3))
    v = np.where(bad[:, None, :, None], 0.0, v)
    scale = np.maximum((np.abs(v).max(axis=(1, 3)) / 448.0).astype(np.float32), np.float32(2.0 ** -126))
    q = (v / scale.astype(np.float64)[:, None, :, None]).astype(np.float32).astype(np.float64)
    byte = nearest_even(np.abs(q), E4M3) + 128 * np.signbit(q)
    byte = byte.reshape(v.shape[0] * block_rows, -1)[:rows, :cols].astype(np.uint8)
    return byte, np.where(bad, np.float32(np.nan), scale).T.astype(np.float32)


def values(byte: np.ndarray, scale: np.ndarray, block_rows: int) -> np.ndarray:
    """code * scale of every element [rows, cols]."""
    mag = np.append(E4M3, np.nan)[byte & 127]
    rows, cols = byte.shape
    s = scale.T.astype(np.float64).repeat(block_rows, axis=0)[:rows].repeat(BLOCK, axis=1)[:, :cols]
    return np.where(byte >= 128, -mag, mag) * s


def pad_codes(byte: np.ndarray) -> np.ndarray:
    """[rows, cols] -> [rows, cols rounded up to 16], zeros behind the last column."""
    return np.pad(byte, ((0, 0), (0, -byte.shape[1] % 16)))


def gemm(a: np.ndarray, b: np.ndarray, alpha: float = 1.0, bias: Optional[np.ndarray] = None) -> np.ndarray:
    """alpha * a b^T + bias of operands' values a [M, K], b [N, K]."""
    d = alpha * (a @ b.T)
    return d if bias is None else d + bias.astype(np.float64)


def residual_rms(x: np.ndarray, residual: Optional[np.ndarray], gamma: np.ndarray, beta: Optional[np.ndarray], eps: float,
                 silu: bool) -> Tuple[np.ndarray, np.ndarray]:
    """(h, y): h = x + residual, y = h / sqrt(mean h^2 + eps) * gamma + beta, then SiLU."""
    h = x if residual is None else x + residual
    y = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps) * gamma
    if beta is not None:
        y = y + beta
    return h, y / (1.0 + np.exp(-y)) if silu else y
