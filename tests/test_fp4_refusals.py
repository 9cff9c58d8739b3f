"""Sizes and refusals of the 4-bit entry points, and the binding's struct layouts.  No GPU: a refused call returns before
anything is enqueued, so the pointers here are never followed."""
import ctypes as C
import os
import shutil
import subprocess

import pytest

from patch_tiled_causal_gb300 import build, vaedec as vd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # a 16-byte aligned number in the place of a pointer


@pytest.fixture(scope="module")
def lib():
    build.build()
    return vd.load()


@pytest.mark.parametrize("rows,cols", [(0, 1), (1, 1), (127, 32), (128, 33), (129, 128), (300, 1000), (3520, 1024)])
def test_buffer_sizes(lib, rows, cols):
    assert lib.vae_fp4_codes_bytes(rows, cols) == rows * (-(-cols // 32) * 16)
    for fmt, blk in ((vd.VAE_MXFP4, 32), (vd.VAE_NVFP4, 16)):
        nb = -(-cols // blk)
        assert lib.vae_fp4_scales_bytes(fmt, rows, cols) == -(-rows // 128) * -(-nb // 4) * 512


def test_buffer_sizes_of_nonsense_are_zero(lib):
    assert lib.vae_fp4_codes_bytes(-1, 8) == 0 and lib.vae_fp4_codes_bytes(8, 0) == 0
    assert lib.vae_fp4_scales_bytes(2, 8, 8) == 0 and lib.vae_fp4_scales_bytes(vd.VAE_MXFP4, -1, 8) == 0
    assert lib.vae_fp4_scales_bytes(vd.VAE_MXFP4, 8, 0) == 0
    assert lib.vae_fp4_codes_bytes(1 << 33, 64) == (1 << 33) * 32  # beyond 32 bits


GOOD = dict(rows=8, ld=64, cols=64, format=vd.VAE_MXFP4, dtype=vd.VAE_BF16, tensor_scale=1.0)


def desc(**kw):
    return vd.VaeFp4Desc(**{**GOOD, **kw})


BAD_DESC = [
    (dict(format=2), vd.VAE_ERR_INVALID_ARG), (dict(format=-1), vd.VAE_ERR_INVALID_ARG),
    (dict(dtype=vd.VAE_FP8), vd.VAE_ERR_INVALID_ARG), (dict(dtype=vd.VAE_FP32_TC), vd.VAE_ERR_INVALID_ARG),
    (dict(tensor_scale=0.5), vd.VAE_ERR_INVALID_ARG),  # MXFP4 has none
    (dict(format=vd.VAE_NVFP4, tensor_scale=0.0), vd.VAE_ERR_INVALID_ARG),
    (dict(format=vd.VAE_NVFP4, tensor_scale=-1.0), vd.VAE_ERR_INVALID_ARG),
    (dict(format=vd.VAE_NVFP4, tensor_scale=float("nan")), vd.VAE_ERR_INVALID_ARG),
    (dict(format=vd.VAE_NVFP4, tensor_scale=float("inf")), vd.VAE_ERR_INVALID_ARG),
    (dict(format=vd.VAE_NVFP4, tensor_scale=1e-30), vd.VAE_ERR_INVALID_ARG),
    (dict(rows=-1), vd.VAE_ERR_INVALID_ARG), (dict(cols=0), vd.VAE_ERR_INVALID_ARG), (dict(ld=63), vd.VAE_ERR_INVALID_ARG),
    (dict(cols=262145, ld=262145), vd.VAE_ERR_UNSUPPORTED), (dict(rows=1 << 40), vd.VAE_ERR_UNSUPPORTED),
    (dict(ld=(1 << 32) + 1), vd.VAE_ERR_UNSUPPORTED), (dict(rows=1 << 31, cols=1, ld=1), vd.VAE_ERR_UNSUPPORTED), (dict(rows=1 << 30, cols=2048, ld=2048), vd.VAE_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", BAD_DESC)
def test_quantize_and_dequantize_refuse(lib, kw, code):
    d = desc(**kw)
    assert lib.vae_quantize_fp4(P, P, P, C.byref(d), None) == code
    assert lib.vae_dequantize_fp4(P, P, P, C.byref(d), None) == code


def test_quantize_and_dequantize_pointers(lib):
    d = desc()
    for f in (lib.vae_quantize_fp4, lib.vae_dequantize_fp4):
        assert f(P, P, P, None, None) == vd.VAE_ERR_INVALID_ARG
        for k in range(3):
            args = [P, P, P]
            args[k] = None
            assert f(*args, C.byref(d), None) == vd.VAE_ERR_INVALID_ARG
    assert lib.vae_quantize_fp4(P + 1, P, P, C.byref(d), None) == vd.VAE_ERR_ALIGNMENT
    assert lib.vae_quantize_fp4(P, P + 8, P, C.byref(d), None) == vd.VAE_ERR_ALIGNMENT
    assert lib.vae_quantize_fp4(P, P, P + 4, C.byref(d), None) == vd.VAE_ERR_ALIGNMENT
    assert lib.vae_dequantize_fp4(P, P, P + 1, C.byref(d), None) == vd.VAE_ERR_ALIGNMENT
    assert lib.vae_dequantize_fp4(P + 8, P, P, C.byref(d), None) == vd.VAE_ERR_ALIGNMENT
    empty = desc(rows=0)  # nothing to do, whatever the pointers
    assert lib.vae_quantize_fp4(None, None, None, C.byref(empty), None) == vd.VAE_OK
    assert lib.vae_dequantize_fp4(None, None, None, C.byref(empty), None) == vd.VAE_OK


GEMM = dict(M=8, N=16, K=64, ld_d=16, format=vd.VAE_NVFP4, out_dtype=vd.VAE_BF16, alpha=1.0)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), vd.VAE_ERR_INVALID_ARG), (dict(N=0), vd.VAE_ERR_INVALID_ARG), (dict(K=0), vd.VAE_ERR_INVALID_ARG),
    (dict(ld_d=15), vd.VAE_ERR_INVALID_ARG), (dict(format=3), vd.VAE_ERR_INVALID_ARG),
    (dict(out_dtype=vd.VAE_FP8), vd.VAE_ERR_INVALID_ARG), (dict(K=262145), vd.VAE_ERR_UNSUPPORTED),
    (dict(M=(1 << 30) + 1), vd.VAE_ERR_UNSUPPORTED), (dict(ld_d=(1 << 32) + 1), vd.VAE_ERR_UNSUPPORTED),
    (dict(M=1 << 30, N=1 << 30, ld_d=1 << 30), vd.VAE_ERR_UNSUPPORTED),
])
def test_gemm_refuses(lib, kw, code):
    d = vd.VaeFp4GemmDesc(**{**GEMM, **kw})
    assert lib.vae_gemm_fp4(P, P, P, P, None, P, C.byref(d), None) == code


def test_gemm_pointers(lib):
    d = vd.VaeFp4GemmDesc(**GEMM)
    assert lib.vae_gemm_fp4(P, P, P, P, None, P, None, None) == vd.VAE_ERR_INVALID_ARG
    for k in (0, 1, 2, 3, 5):
        args = [P, P, P, P, None, P]
        args[k] = None
        assert lib.vae_gemm_fp4(*args, C.byref(d), None) == vd.VAE_ERR_INVALID_ARG
        args[k] = P + (8 if k < 4 else 1)
        assert lib.vae_gemm_fp4(*args, C.byref(d), None) == vd.VAE_ERR_ALIGNMENT
    assert lib.vae_gemm_fp4(P, P, P, P, P + 2, P, C.byref(d), None) == vd.VAE_ERR_ALIGNMENT
    d.M = 0
    assert lib.vae_gemm_fp4(None, None, None, None, None, None, C.byref(d), None) == vd.VAE_OK


def test_norms_refuse(lib):
    def gn(fmt=vd.VAE_MXFP4, ts=1.0, B=1, T=1, C_=64, groups=8, scales=P, codes=P, **kw):
        d = vd.gn_desc(B, T, 4, 4, C_, groups, [0, 4], [0, 4], **kw)
        return lib.vae_patch_groupnorm_silu_fp4(P, P, P, codes, scales, P, C.byref(d), fmt, ts, None)

    assert gn(fmt=2) == vd.VAE_ERR_INVALID_ARG and gn(ts=2.0) == vd.VAE_ERR_INVALID_ARG
    assert gn(fmt=vd.VAE_NVFP4, ts=0.0) == vd.VAE_ERR_INVALID_ARG
    assert gn(C_=48, groups=6) == vd.VAE_ERR_UNSUPPORTED
    assert gn(B=2, T=40000) == vd.VAE_ERR_UNSUPPORTED
    assert gn(scales=P + 8) == vd.VAE_ERR_ALIGNMENT and gn(codes=P + 8) == vd.VAE_ERR_ALIGNMENT
    assert gn(scales=None) == vd.VAE_ERR_INVALID_ARG
    assert gn(in_dtype=vd.VAE_FP8) == vd.VAE_ERR_INVALID_ARG

    def rms(fmt=vd.VAE_MXFP4, ts=1.0, B=1, T=1, H=4, W=4, C_=64, scales=P, codes=P, in_dtype=vd.VAE_BF16):
        d = vd.VaeRmsDesc(B, T, H, W, C_, 1e-6, 1, in_dtype, vd.VAE_BF16)
        return lib.vae_channel_rmsnorm_silu_fp4(P, P, P, codes, scales, C.byref(d), fmt, ts, None)

    assert rms(fmt=2) == vd.VAE_ERR_INVALID_ARG and rms(ts=0.5) == vd.VAE_ERR_INVALID_ARG
    assert rms(C_=16) == vd.VAE_ERR_UNSUPPORTED and rms(C_=96) == vd.VAE_ERR_UNSUPPORTED and rms(C_=2048) == vd.VAE_ERR_UNSUPPORTED
    assert rms(T=1024, H=1024, W=1024) == vd.VAE_ERR_UNSUPPORTED
    assert rms(B=0) == vd.VAE_ERR_INVALID_ARG and rms(in_dtype=vd.VAE_FP8) == vd.VAE_ERR_INVALID_ARG
    assert rms(scales=P + 8) == vd.VAE_ERR_ALIGNMENT and rms(codes=None) == vd.VAE_ERR_INVALID_ARG


def test_binding_refuses_host_tensors_and_wrong_shapes(lib):
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 32)
    with pytest.raises(ValueError):
        vd.quantize_fp4(x, x, x, vd.VAE_MXFP4)  # not on a GPU
    with pytest.raises(ValueError):
        vd.fp4_empty(4, 0, vd.VAE_MXFP4, device="cpu")
    with pytest.raises(ValueError):
        vd.fp4_empty(4, 32, 5, device="cpu")
    c, s = vd.fp4_empty(130, 40, vd.VAE_NVFP4, device="cpu")
    assert c.shape == (130, 32) and s.numel() == 2 * 512


@pytest.mark.parametrize("py,name", [("VaeFp4Desc", "vae_fp4_desc_t"), ("VaeFp4GemmDesc", "vae_fp4_gemm_desc_t")])
def test_struct_layouts(tmp_path, py, name):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    cls = getattr(vd, py)
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "vaedec.h"', "int main(void) {",
             f'  printf("%zu\\n", sizeof({name}));']
    lines += [f'  printf("%zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_] + ["  return 0;", "}"]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines) + "\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [C.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_]


class Shape:
    """A CUDA tensor's metadata without its memory: what the binding asks before it makes a call."""
    def __init__(self, dtype, *shape):
        self.dtype, self.shape, self.device, self.is_cuda = dtype, shape, "cuda:0", True

    def get_device(self):
        return 0

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for v in self.shape:
            n *= v
        return n

    def stride(self):
        return tuple(Shape(self.dtype, *self.shape[i + 1:]).numel() for i in range(len(self.shape)))

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return P


@pytest.mark.parametrize("M,N,K", [((1 << 32) + 5, 16, 64), (8, (1 << 32) + 16, 64), (8, 16, (1 << 32) + 64), (1 << 31, 16, 64),
                                   (8, 16, (1 << 33) + 96)])
def test_products_refuse_sizes_beyond_c_ints(lib, monkeypatch, M, N, K):
    """Sizes whose low 32 bits alone would pass for others.  (Reaching the call is the failure: nothing is enqueued here.)"""
    torch = pytest.importorskip("torch")

    def reached(*args):
        pytest.fail(f"the call is made: {args}")

    monkeypatch.setattr(vd, "_call_on", reached)
    monkeypatch.setattr(vd, "_stream", lambda s: None)
    monkeypatch.setattr(lib, "vae_gemm_bf16", reached)
    pitch, u8 = (K + 31) // 32 * 16, torch.uint8
    a, b = Shape(u8, M, pitch), Shape(u8, N, pitch)
    sa, sb = [Shape(u8, (r + 127) // 128 * ((K + 63) // 64) * 512) for r in (M, N)]
    with pytest.raises(ValueError, match="C ints"):
        vd.gemm_fp4(a, sa, b, sb, Shape(torch.bfloat16, M, N), K, vd.VAE_NVFP4)
    with pytest.raises(ValueError, match="C ints"):
        vd.gemm_bf16(Shape(torch.bfloat16, 1, M, K), Shape(torch.bfloat16, 1, N, K), Shape(torch.bfloat16, 1, M, N))


def test_empty_operand_refuses_columns_beyond_c_ints(lib):
    pytest.importorskip("torch")
    with pytest.raises(ValueError, match="C ints"):
        vd.fp4_empty(1, (1 << 32) + 32, vd.VAE_MXFP4, device="cpu")
