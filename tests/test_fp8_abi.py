"""Refusals of the 8-bit operators, without a GPU: every call fails its checks before any CUDA call."""
import pytest
import torch

import microscaling_fp4_quantization_mxfp4_b200 as fp
from microscaling_fp4_quantization_mxfp4_b200 import _lib, build

FAKE = 0x10000            # 16-byte aligned, never dereferenced
ARG, SHAPE, ALIGN = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_scales_bytes(lib):
    assert lib.fp4_fp8_scales_bytes(130, 640, 1, 0) == 130 * 5
    assert lib.fp4_fp8_scales_bytes(130, 640, 1, 1) == 256 * 8
    assert lib.fp4_fp8_scales_bytes(129, 136, 0, 0) == 136 * 2          # axis 0: [cols, ceil(rows / 128)]
    assert lib.fp4_fp8_scales_bytes(1, 1, 1, 1) == 512
    for bad in ((0, 8, 1, 0), (8, 0, 1, 0), (8, 8, 2, 0), (8, 8, 1, 2)):
        assert lib.fp4_fp8_scales_bytes(*bad) == 0


def _changed(good, changes):
    for at, value, status in changes:
        args = list(good)
        args[at] = value
        yield args, status


def test_quantize_refusals(lib):
    # x, rows, cols, ld, fmt, axis, codes, ldc, scales, sf_layout, stream
    good = (FAKE, 4, 64, 64, 0, 1, FAKE, 64, FAKE, 1, None)
    for args, status in _changed(good, [
            (0, None, ARG), (1, 0, ARG), (2, 0, ARG), (2, 60, SHAPE), (3, 56, ARG), (3, 68, SHAPE), (0, FAKE + 8, ALIGN),
            (4, 2, ARG), (4, -1, ARG), (5, 2, ARG), (6, None, ARG), (6, FAKE + 8, ALIGN), (7, 48, ARG), (7, 72, ALIGN),
            (8, None, ARG), (8, FAKE + 2, ALIGN), (9, 2, ARG), (1, 1 << 31, SHAPE)]):
        assert lib.fp4_fp8_quantize(*args) == status, args
    # axis 0: the row stride of the codes is at least the number of rows; tiles are counted in 32 bits
    assert lib.fp4_fp8_quantize(FAKE, 100, 64, 64, 0, 0, FAKE, 96, FAKE, 1, None) == ARG
    assert lib.fp4_fp8_quantize(FAKE, (1 << 31) - 16, 16384, 16384, 0, 0, FAKE, 1 << 31, FAKE, 1, None) == SHAPE


def test_quantize_2d_refusals(lib):
    # x, rows, cols, ld, fmt, codes, ldc, scales, codes_t, ldc_t, scales_t, sf_layout, stream
    good = (FAKE, 32, 64, 64, 0, FAKE, 64, FAKE, FAKE, 32, FAKE, 1, None)
    for args, status in _changed(good, [
            (0, None, ARG), (0, FAKE + 2, ALIGN), (2, 60, SHAPE), (4, 5, ARG), (5, None, ARG), (6, 65, ALIGN),
            (7, None, ARG), (8, None, ARG), (10, None, ARG), (8, FAKE + 4, ALIGN), (9, 16, ARG), (9, 40, ALIGN),
            (10, FAKE + 1, ALIGN), (11, 7, ARG), (1, 0, ARG)]):
        assert lib.fp4_fp8_quantize_2d(*args) == status, args


def test_dequantize_refusals(lib):
    # codes, ldc, scales, rows, cols, fmt, sf_layout, out, out_dtype, stream
    good = (FAKE, 64, FAKE, 4, 64, 0, 0, FAKE, 0, None)
    for args, status in _changed(good, [
            (0, None, ARG), (0, FAKE + 8, ALIGN), (1, 48, ARG), (1, 72, ALIGN), (2, None, ARG), (3, 0, ARG), (4, 0, ARG),
            (5, 3, ARG), (6, 2, ARG), (7, None, ARG), (7, FAKE + 4, ALIGN), (8, 2, ARG), (3, 1 << 31, SHAPE)]):
        assert lib.fp4_fp8_dequantize(*args) == status, args


def test_gemm_refusals(lib):
    # a, lda, a_sf, b, ldb, b_sf, M, N, K, a_fmt, b_fmt, y, ldy, y_dtype, stream
    good = (FAKE, 112, FAKE, FAKE, 112, FAKE, 4, 8, 100, 0, 1, FAKE, 8, 1, None)
    for args, status in _changed(good, [
            (0, None, ARG), (0, FAKE + 8, ALIGN), (1, 96, ARG), (1, 120, ALIGN), (2, None, ARG), (2, FAKE + 4, ALIGN),
            (3, None, ARG), (4, 100, ALIGN), (4, 1 << 40, SHAPE), (5, FAKE + 8, ALIGN), (6, 0, ARG), (7, 0, ARG), (8, 0, ARG), (8, 113, ARG),
            (9, 2, ARG), (10, -1, ARG), (11, None, ARG), (11, FAKE + 1, ALIGN), (12, 7, ARG), (13, 2, ARG),
            (6, 1 << 31, SHAPE)]):
        assert lib.fp4_fp8_gemm(*args) == status, args
    # scale atoms, 128 rows x 512 elements of K, are counted in 32 bits
    big = list(good)
    big[1], big[4], big[6], big[8] = 1 << 26, 1 << 26, 1 << 22, 1 << 26
    assert lib.fp4_fp8_gemm(*big) == SHAPE
    assert lib.fp4_fp8_gemm(*good[:11], FAKE + 2, 8, 0, None) == ALIGN          # fp32 output on a 2-byte boundary


def test_rmsnorm_refusals(lib):
    # x, ldx, residual, ldr, weight, wdtype, rows, cols, eps, fmt, codes, ldc, scales, sf, residual_out, rstd, norm_out, stream
    good = (FAKE, 64, FAKE, 64, FAKE, 1, 4, 64, 1e-6, 0, FAKE, 64, FAKE, 1, FAKE, FAKE, FAKE, None)
    for args, status in _changed(good, [
            (0, None, ARG), (0, FAKE + 2, ALIGN), (1, 56, ARG), (1, 68, SHAPE), (2, None, ARG), (2, FAKE + 8, ALIGN),
            (3, 32, ARG), (4, None, ARG), (4, FAKE + 8, ALIGN), (5, 2, ARG), (6, 0, ARG), (6, 1 << 31, SHAPE), (7, 0, ARG),
            (7, 60, SHAPE), (7, 16392, SHAPE), (8, -1.0, ARG), (8, float("nan"), ARG), (8, float("inf"), ARG), (9, 2, ARG),
            (10, None, ARG), (11, 72, ALIGN), (12, None, ARG), (12, FAKE + 1, ALIGN), (13, 3, ARG), (14, None, ARG),
            (14, FAKE + 2, ALIGN), (15, FAKE + 2, ALIGN), (16, FAKE + 2, ALIGN)]):
        assert lib.fp4_rmsnorm_fp8_quantize(*args) == status, args
    no_residual = list(good)
    no_residual[2] = None
    assert lib.fp4_rmsnorm_fp8_quantize(*no_residual) == ARG            # residual_out without a residual


def test_rmsnorm_backward_refusals(lib):
    # dy, lddy, h, ldh, weight, wdtype, rstd, dres, lddr, rows, cols, dx, dweight, workspace, bytes, stream
    good = (FAKE, 64, FAKE, 64, FAKE, 1, FAKE, FAKE, 64, 4, 64, FAKE, FAKE, FAKE, 1 << 30, None)
    for args, status in _changed(good, [
            (0, None, ARG), (0, FAKE + 2, ALIGN), (1, 32, ARG), (1, 68, SHAPE), (2, None, ARG), (3, 32, ARG), (4, None, ARG),
            (4, FAKE + 4, ALIGN), (5, 9, ARG), (6, None, ARG), (6, FAKE + 2, ALIGN), (7, FAKE + 4, ALIGN), (8, 32, ARG),
            (9, 0, ARG), (10, 12, SHAPE), (10, 16392, SHAPE), (11, None, ARG), (11, FAKE + 8, ALIGN), (12, None, ARG),
            (12, FAKE + 8, ALIGN), (13, None, ARG), (13, FAKE + 8, ALIGN)]):
        assert lib.fp4_rmsnorm_backward(*args) == status, args
    for bad in ((0, 64), (4, 0), (4, 12), (4, 16392)):
        assert lib.fp4_rmsnorm_backward_workspace(*bad) == 0


def test_binding_needs_cuda_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    u8 = torch.zeros(4, 64, dtype=torch.uint8)
    for call in (lambda: fp.fp4_fp8_quantize(x), lambda: fp.fp4_fp8_quantize_2d(x), lambda: fp.fp4_fp8_dequantize(u8, u8),
                 lambda: fp.fp4_fp8_gemm(u8, u8, u8, u8), lambda: fp.fp4_rmsnorm_fp8_quantize(x, x[0]),
                 lambda: fp.fp4_rmsnorm_backward(x, x, x[0], x[:, 0].float())):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_exported():
    for name in ("E4M3", "E5M2", "Fp8Quantized", "Fp8RmsNorm", "fp4_fp8_quantize", "fp4_fp8_quantize_2d", "fp4_fp8_dequantize",
                 "fp4_fp8_gemm", "fp4_fp8_scales_bytes", "fp4_rmsnorm_fp8_quantize", "fp4_rmsnorm_backward"):
        assert name in fp.__all__ and hasattr(fp, name)
