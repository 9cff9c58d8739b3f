"""Sizes and refusals of the 8-bit block-scaled entry points, and the binding's struct layouts.  No GPU: a refused call
returns before anything is enqueued, so the pointers here are never followed."""
import ctypes as C
import os
import shutil
import subprocess

import pytest
import torch

from patch_tiled_causal_gb300 import build, vaedec as vd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # a 16-byte aligned number in the place of a pointer
INVALID, UNSUPPORTED, ALIGNMENT = vd.VAE_ERR_INVALID_ARG, vd.VAE_ERR_UNSUPPORTED, vd.VAE_ERR_ALIGNMENT


@pytest.fixture(scope="module")
def lib():
    build.build()
    return vd.load()


@pytest.mark.parametrize("rows,cols", [(0, 1), (1, 1), (127, 16), (128, 17), (129, 128), (300, 1000), (3520, 1024)])
def test_buffer_sizes(lib, rows, cols):
    assert lib.vae_fp8_codes_bytes(rows, cols) == rows * (-(-cols // 16) * 16)
    for br in (1, 128):
        assert lib.vae_fp8_scales_bytes(rows, cols, br) == -(-rows // br) * -(-cols // 128) * 4
        codes, scales = vd.fp8_empty(rows, cols, br, device="cpu")
        assert codes.numel() == lib.vae_fp8_codes_bytes(rows, cols)
        assert 4 * scales.numel() == lib.vae_fp8_scales_bytes(rows, cols, br)


def test_buffer_sizes_of_nonsense(lib):
    assert lib.vae_fp8_codes_bytes(-1, 8) == 0 and lib.vae_fp8_codes_bytes(8, 0) == 0
    assert lib.vae_fp8_scales_bytes(8, 8, 2) == 0 and lib.vae_fp8_scales_bytes(-1, 8, 1) == 0
    assert lib.vae_fp8_scales_bytes(8, -8, 128) == 0
    assert lib.vae_fp8_codes_bytes(1 << 33, 64) == 1 << 39  # beyond 32 bits
    for bad in ((-1, 8, 1), (8, 0, 1), (8, 8, 64), (8, 1 << 31, 1)):
        with pytest.raises(ValueError):
            vd.fp8_empty(*bad, device="cpu")


GOOD = dict(rows=8, ld=64, cols=64, block_rows=1, dtype=vd.VAE_BF16)


@pytest.mark.parametrize("kw,code", [
    (dict(block_rows=0), INVALID), (dict(block_rows=64), INVALID), (dict(block_rows=-1), INVALID),
    (dict(dtype=vd.VAE_FP8), INVALID), (dict(dtype=vd.VAE_FP32_TC), INVALID), (dict(dtype=9), INVALID),
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(cols=-3), INVALID), (dict(ld=63), INVALID), (dict(ld=-64), INVALID),
    (dict(cols=262145, ld=262145), UNSUPPORTED), (dict(rows=1 << 40), UNSUPPORTED), (dict(ld=(1 << 32) + 1), UNSUPPORTED),
    (dict(rows=1 << 31, cols=1, ld=1), UNSUPPORTED), (dict(rows=1 << 30, cols=2048, ld=2048), UNSUPPORTED),
])
def test_quantize_and_dequantize_refuse(lib, kw, code):
    d = vd.VaeFp8Desc(**{**GOOD, **kw})
    assert lib.vae_quantize_fp8(P, P, P, C.byref(d), None) == code
    assert lib.vae_dequantize_fp8(P, P, P, C.byref(d), None) == code


def test_quantize_and_dequantize_pointers(lib):
    d = vd.VaeFp8Desc(**GOOD)
    for f in (lib.vae_quantize_fp8, lib.vae_dequantize_fp8):
        assert f(P, P, P, None, None) == INVALID
        for k in range(3):
            args = [P, P, P]
            args[k] = None
            assert f(*args, C.byref(d), None) == INVALID
    for k, off in ((0, 1), (1, 8), (2, 2)):  # x, codes, scales
        args = [P, P, P]
        args[k] += off
        assert lib.vae_quantize_fp8(*args, C.byref(d), None) == ALIGNMENT
    for k, off in ((0, 8), (1, 2), (2, 1)):  # codes, scales, y
        args = [P, P, P]
        args[k] += off
        assert lib.vae_dequantize_fp8(*args, C.byref(d), None) == ALIGNMENT
    d.rows = 0  # nothing to do, whatever the pointers
    assert lib.vae_quantize_fp8(None, None, None, C.byref(d), None) == vd.VAE_OK
    assert lib.vae_dequantize_fp8(None, None, None, C.byref(d), None) == vd.VAE_OK


GEMM = dict(M=8, N=16, K=64, ld_d=16, out_dtype=vd.VAE_BF16, alpha=1.0)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(ld_d=15), INVALID),
    (dict(out_dtype=vd.VAE_FP8), INVALID), (dict(out_dtype=vd.VAE_FP32_TC), INVALID), (dict(K=262145), UNSUPPORTED),
    (dict(M=(1 << 30) + 1), UNSUPPORTED), (dict(N=(1 << 30) + 1, ld_d=1 << 31), UNSUPPORTED),
    (dict(ld_d=(1 << 32) + 1), UNSUPPORTED), (dict(M=1 << 30, N=1 << 30, ld_d=1 << 30), UNSUPPORTED),
])
def test_gemm_refuses(lib, kw, code):
    d = vd.VaeFp8GemmDesc(**{**GEMM, **kw})
    assert lib.vae_gemm_fp8(P, P, P, P, None, P, C.byref(d), None) == code


def test_gemm_pointers(lib):
    d = vd.VaeFp8GemmDesc(**GEMM)
    assert lib.vae_gemm_fp8(P, P, P, P, None, P, None, None) == INVALID
    for k, off in ((0, 8), (1, 2), (2, 8), (3, 1), (5, 1)):
        args = [P, P, P, P, None, P]
        args[k] = None
        assert lib.vae_gemm_fp8(*args, C.byref(d), None) == INVALID
        args[k] = P + off
        assert lib.vae_gemm_fp8(*args, C.byref(d), None) == ALIGNMENT
    assert lib.vae_gemm_fp8(P, P, P, P, P + 2, P, C.byref(d), None) == ALIGNMENT
    d.M = 0
    assert lib.vae_gemm_fp8(None, None, None, None, None, None, C.byref(d), None) == vd.VAE_OK


RMS = dict(rows=8, ld_x=64, ld_residual=64, ld_total=64, cols=64, eps=1e-6, silu=0, dtype=vd.VAE_BF16, residual_dtype=vd.VAE_FP32)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=vd.VAE_FP8), INVALID), (dict(residual_dtype=vd.VAE_FP8), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(ld_x=63), INVALID),
    (dict(ld_residual=63), INVALID), (dict(ld_total=63), INVALID), (dict(ld_x=(1 << 32) + 1), UNSUPPORTED),
    (dict(ld_residual=(1 << 32) + 1), UNSUPPORTED), (dict(ld_total=(1 << 32) + 1), UNSUPPORTED),
    (dict(cols=32769, ld_x=32769, ld_residual=32769, ld_total=32769), UNSUPPORTED), (dict(rows=1 << 40), UNSUPPORTED),
])
def test_rms_refuses(lib, kw, code):
    d = vd.VaeFp8RmsDesc(**{**RMS, **kw})
    assert lib.vae_residual_rmsnorm_silu_fp8(P, P, P, P, P, P, P, C.byref(d), None) == code


def test_rms_pointers(lib):
    f, d = lib.vae_residual_rmsnorm_silu_fp8, vd.VaeFp8RmsDesc(**RMS)
    assert f(P, P, P, P, P, P, P, None, None) == INVALID
    for k in (0, 2, 5, 6):  # x, gamma, codes, scales (residual, beta and total may be null)
        args = [P] * 7
        args[k] = None
        assert f(*args, C.byref(d), None) == INVALID
    for k, off in enumerate((1, 2, 2, 2, 2, 8, 2)):
        args = [P] * 7
        args[k] += off
        assert f(*args, C.byref(d), None) == ALIGNMENT
    d.rows = 0
    assert f(None, None, None, None, None, None, None, C.byref(d), None) == vd.VAE_OK


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x, codes = torch.zeros(4, 32), torch.zeros(4, 32, dtype=torch.float8_e4m3fn)
    scales = torch.zeros(1, 4)
    for call in (lambda: vd.quantize_fp8(x, codes, scales), lambda: vd.dequantize_fp8(codes, scales, x),
                 lambda: vd.gemm_fp8(codes, scales, codes, scales, x, 32),
                 lambda: vd.residual_rmsnorm_silu_fp8(x, None, x[0], None, None, codes, scales)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("py,c", [("VaeFp8Desc", "vae_fp8_desc_t"), ("VaeFp8GemmDesc", "vae_fp8_gemm_desc_t"),
                                  ("VaeFp8RmsDesc", "vae_fp8_rms_desc_t")])
def test_binding_structs_match_header(tmp_path, py, c):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    cls = getattr(vd, py)
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "vaedec.h"', "int main(void) {",
             f'  printf("%zu\\n", sizeof({c}));'] + [f'  printf("%zu\\n", offsetof({c}, {n}));' for n, _ in cls._fields_]
    (tmp_path / "l.c").write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run([cc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"), "-o", str(tmp_path / "l")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "l")], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [C.sizeof(cls)] + [getattr(cls, n).offset for n, _ in cls._fields_]
