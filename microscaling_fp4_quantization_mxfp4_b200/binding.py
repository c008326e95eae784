"""Thin Python binding of libfp4 (include/fp4.h), one function per C entry point.

Argument marshalling only: tensors are checked for device, dtype and layout,
output buffers are allocated with PyTorch when the caller gives none, and the
raw pointers plus the current CUDA stream go to the C ABI.  Every step of the
computation runs in the library's CUDA kernels; there is no CPU path, and
every call raises if libfp4.so is missing or a tensor is not on a GPU.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib

MXFP4, NVFP4, NVFP4_4O6, MXFP4_GS = 0, 1, 2, 3
RTN, SR = 0, 1
SF_ROWMAJOR, SF_MMA = 0, 1
OUT_F32, OUT_BF16 = 0, 1

_FMT = {"mxfp4": MXFP4, "nvfp4": NVFP4, "nvfp4_4o6": NVFP4_4O6, "mxfp4_gs": MXFP4_GS,
        MXFP4: MXFP4, NVFP4: NVFP4, NVFP4_4O6: NVFP4_4O6, MXFP4_GS: MXFP4_GS}
_RND = {"rtn": RTN, "sr": SR, RTN: RTN, SR: SR}
_SF = {"rowmajor": SF_ROWMAJOR, "mma": SF_MMA, SF_ROWMAJOR: SF_ROWMAJOR, SF_MMA: SF_MMA}
_OUT = {"f32": OUT_F32, "bf16": OUT_BF16, torch.float32: OUT_F32, torch.bfloat16: OUT_BF16,
        OUT_F32: OUT_F32, OUT_BF16: OUT_BF16}
E4M3, E5M2 = 0, 1
_FMT8 = {"e4m3": E4M3, "e5m2": E5M2, torch.float8_e4m3fn: E4M3, torch.float8_e5m2: E5M2, E4M3: E4M3, E5M2: E5M2}
_CODE8 = ((torch.uint8, torch.float8_e4m3fn), (torch.uint8, torch.float8_e5m2))      # by format
_SCALE8 = (torch.uint8, torch.float8_e8m0fnu)
FP8_BLOCK = 128
BLOCK = {MXFP4: 32, NVFP4: 16, NVFP4_4O6: 16, MXFP4_GS: 32}


class Fp4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.load().fp4_status_string(status).decode()
        super().__init__(f"{where}: {msg} (status {status})")


class Fp4Quantized(NamedTuple):
    codes: torch.Tensor          # uint8 [out_rows, L/2]
    scales: torch.Tensor         # uint8, row-major [out_rows, L/block] or flat tensor-core layout
    tensor_scale: Optional[torch.Tensor]   # fp32 [1] (NVFP4) or None


class Fp8Quantized(NamedTuple):
    codes: torch.Tensor          # uint8 [out_rows, L], rows a multiple of 16 bytes apart
    scales: torch.Tensor         # uint8, row-major [out_rows, ceil(L / 128)] or flat tensor-core layout


class Fp8RmsNorm(NamedTuple):
    codes: torch.Tensor                    # as Fp8Quantized
    scales: torch.Tensor
    residual_out: Optional[torch.Tensor]   # bf16 x + residual, or None without a residual
    rstd: torch.Tensor                     # fp32 [rows]


def _check(status: int, where: str) -> None:
    if status != 0:
        raise Fp4Error(status, where)


def _stream(stream) -> int:
    """cudaStream_t of `stream`, or of the current device's current stream (read as a raw handle,
    without building a Stream object)."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _need_cuda(t: torch.Tensor, name: str) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (libfp4 has no CPU path)")


def _bf16_matrix(x: torch.Tensor, name: str = "x") -> None:
    _need_cuda(x, name)
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D bf16 CUDA tensor with unit column stride")


def fp4_codes_bytes(rows: int, cols: int) -> int:
    """Bytes of packed codes for a [rows, cols] tensor (two E2M1 codes per byte); 0 for an empty
    or odd-sized tensor."""
    return _lib.load().fp4_codes_bytes(rows, cols)


def fp4_scales_bytes(rows: int, cols: int, block: int, axis: int, sf_layout="rowmajor") -> int:
    """Bytes of block scales for a [rows, cols] tensor quantized along `axis` in `block`-element
    blocks: one byte per block row-major, or the tensor-core layout padded to 128 rows x 4 block
    columns ("mma"); 0 for an invalid shape."""
    return _lib.load().fp4_scales_bytes(rows, cols, block, axis, _SF[sf_layout])


def fp4_status_string(status: int) -> str:
    """Short message for an fp4_status code (e.g. "invalid argument" for FP4_ERR_ARG)."""
    return _lib.load().fp4_status_string(status).decode()


def fp4_check_device_errors(stream=None) -> None:
    """Synchronize and raise if a bounded device wait expired since the last check."""
    _check(_lib.load().fp4_check_device_errors(_stream(stream)), "fp4_check_device_errors")


def _alloc_quant_outputs(x, fmt, axis, sf, codes, scales, ts_out):
    rows, cols = x.shape
    orows, qlen = (rows, cols) if axis == 1 else (cols, rows)
    if codes is None:
        codes = torch.empty((orows, qlen // 2), dtype=torch.uint8, device=x.device)
    if scales is None:
        nbytes = fp4_scales_bytes(rows, cols, BLOCK[fmt], axis, sf)
        if nbytes == 0:
            raise ValueError("shape not quantizable with this block size along this axis")
        shape = (orows, qlen // BLOCK[fmt]) if sf == SF_ROWMAJOR else (nbytes,)
        scales = torch.empty(shape, dtype=torch.uint8, device=x.device)
    if fmt in (NVFP4, NVFP4_4O6) and ts_out is None:
        ts_out = torch.empty((1,), dtype=torch.float32, device=x.device)
    return codes, scales, ts_out


def fp4_quantize(x: torch.Tensor, fmt="mxfp4", axis: int = 1, rnd="rtn", seed: int = 0,
                 tensor_scale_in: Optional[torch.Tensor] = None, sf_layout="rowmajor", *,
                 codes=None, scales=None, tensor_scale_out=None, first_row: int = 0, stream=None) -> Fp4Quantized:
    """Block-scaled FP4 quantization of a bf16 matrix (see fp4_quantize in include/fp4.h).  With
    first_row > 0, x is a row shard of a larger tensor starting at that row (fp4_quantize_shard)."""
    _bf16_matrix(x)
    f, r, sf = _FMT[fmt], _RND[rnd], _SF[sf_layout]
    codes, scales, ts_out = _alloc_quant_outputs(x, f, axis, sf, codes, scales, tensor_scale_out)
    lib = _lib.load()
    if first_row:
        st = lib.fp4_quantize_shard(
            x.data_ptr(), x.shape[0], x.shape[1], x.stride(0), first_row, f, BLOCK[f], axis, r,
            seed & (2 ** 64 - 1), _ptr(tensor_scale_in), _ptr(ts_out), codes.data_ptr(), scales.data_ptr(), sf,
            _stream(stream))
        _check(st, "fp4_quantize_shard")
    else:
        st = lib.fp4_quantize(
            x.data_ptr(), x.shape[0], x.shape[1], x.stride(0), f, BLOCK[f], axis, r, seed & (2 ** 64 - 1),
            _ptr(tensor_scale_in), _ptr(ts_out), codes.data_ptr(), scales.data_ptr(), sf, _stream(stream))
        _check(st, "fp4_quantize")
    return Fp4Quantized(codes, scales, ts_out if f in (NVFP4, NVFP4_4O6) else None)


def fp4_hadamard_quantize(x: torch.Tensor, had_block: int, fmt="mxfp4", axis: int = 1, rnd="rtn",
                          seed: int = 0, tensor_scale_in=None, sf_layout="rowmajor", *, codes=None,
                          scales=None, tensor_scale_out=None, rotated_out=None, stream=None) -> Fp4Quantized:
    """Block-Hadamard rotation fused ahead of the quantizer (see include/fp4.h)."""
    _bf16_matrix(x)
    f, r, sf = _FMT[fmt], _RND[rnd], _SF[sf_layout]
    codes, scales, ts_out = _alloc_quant_outputs(x, f, axis, sf, codes, scales, tensor_scale_out)
    st = _lib.load().fp4_hadamard_quantize(
        x.data_ptr(), x.shape[0], x.shape[1], x.stride(0), f, BLOCK[f], axis, r, seed & (2 ** 64 - 1),
        _ptr(tensor_scale_in), _ptr(ts_out), codes.data_ptr(), scales.data_ptr(), sf, had_block,
        _ptr(rotated_out), _stream(stream))
    _check(st, "fp4_hadamard_quantize")
    return Fp4Quantized(codes, scales, ts_out if f in (NVFP4, NVFP4_4O6) else None)


def fp4_quantize_dequantize(x: torch.Tensor, fmt="nvfp4", rnd="rtn", seed: int = 0,
                            tensor_scale_in: Optional[torch.Tensor] = None, sf_layout="rowmajor", out_dtype="f32", *,
                            codes=None, scales=None, tensor_scale_out=None, out=None, stream=None):
    """fp4_quantize along rows plus the dequantized values in the same launch (see include/fp4.h).
    Returns (Fp4Quantized, dequantized tensor)."""
    _bf16_matrix(x)
    f, r, sf, od = _FMT[fmt], _RND[rnd], _SF[sf_layout], _OUT[out_dtype]
    codes, scales, ts_out = _alloc_quant_outputs(x, f, 1, sf, codes, scales, tensor_scale_out)
    if out is None:
        out = torch.empty(x.shape, dtype=torch.float32 if od == OUT_F32 else torch.bfloat16, device=x.device)
    st = _lib.load().fp4_quantize_dequantize(
        x.data_ptr(), x.shape[0], x.shape[1], x.stride(0), f, BLOCK[f], r, seed & (2 ** 64 - 1),
        _ptr(tensor_scale_in), _ptr(ts_out), codes.data_ptr(), scales.data_ptr(), sf, out.data_ptr(), od,
        _stream(stream))
    _check(st, "fp4_quantize_dequantize")
    return Fp4Quantized(codes, scales, ts_out if f in (NVFP4, NVFP4_4O6) else None), out


def fp4_quantize_2d(x: torch.Tensor, fmt="nvfp4", rnd="rtn", seed: int = 0,
                    tensor_scale_in: Optional[torch.Tensor] = None, sf_layout="rowmajor", transposed: bool = True,
                    *, codes=None, scales=None, codes_t=None, scales_t=None, tensor_scale_out=None,
                    stream=None):
    """Square-tile (2-D) quantization (see fp4_quantize_2d in include/fp4.h).  Returns
    (W along its rows, W^T along its rows or None) as Fp4Quantized, sharing one tensor scale."""
    _bf16_matrix(x)
    f, r, sf = _FMT[fmt], _RND[rnd], _SF[sf_layout]
    codes, scales, ts_out = _alloc_quant_outputs(x, f, 1, sf, codes, scales, tensor_scale_out)
    if transposed:
        codes_t, scales_t, _ = _alloc_quant_outputs(x, f, 0, sf, codes_t, scales_t, ts_out)
    else:
        codes_t = scales_t = None
    st = _lib.load().fp4_quantize_2d(
        x.data_ptr(), x.shape[0], x.shape[1], x.stride(0), f, BLOCK[f], r, seed & (2 ** 64 - 1),
        _ptr(tensor_scale_in), _ptr(ts_out), codes.data_ptr(), scales.data_ptr(), _ptr(codes_t), _ptr(scales_t),
        sf, _stream(stream))
    _check(st, "fp4_quantize_2d")
    ts = ts_out if f == NVFP4 else None
    return Fp4Quantized(codes, scales, ts), (Fp4Quantized(codes_t, scales_t, ts) if transposed else None)


def fp4_quantize_mse(x: torch.Tensor, rnd="rtn", seed: int = 0, iters: int = 1, sf_layout="rowmajor", *,
                     codes=None, scales=None, tensor_scale_out=None, stream=None) -> Fp4Quantized:
    """NVFP4 quantization along rows with MSE-searched block and tensor scales (see fp4_quantize_mse in
    include/fp4.h); outputs are plain NVFP4."""
    _bf16_matrix(x)
    r, sf = _RND[rnd], _SF[sf_layout]
    codes, scales, ts_out = _alloc_quant_outputs(x, NVFP4, 1, sf, codes, scales, tensor_scale_out)
    st = _lib.load().fp4_quantize_mse(
        x.data_ptr(), x.shape[0], x.shape[1], x.stride(0), NVFP4, 16, r, seed & (2 ** 64 - 1), iters,
        ts_out.data_ptr(), codes.data_ptr(), scales.data_ptr(), sf, _stream(stream))
    _check(st, "fp4_quantize_mse")
    return Fp4Quantized(codes, scales, ts_out)


def fp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, tensor_scale=None, fmt="mxfp4",
                   sf_layout="rowmajor", out_dtype="f32", *, out=None, stream=None) -> torch.Tensor:
    """Codes + scales (+ tensor scale) back to fp32 or bf16 [rows, 2 * codes.shape[1]]."""
    _need_cuda(codes, "codes")
    f, sf, od = _FMT[fmt], _SF[sf_layout], _OUT[out_dtype]
    rows, cols = codes.shape[0], codes.shape[1] * 2
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.float32 if od == OUT_F32 else torch.bfloat16,
                          device=codes.device)
    st = _lib.load().fp4_dequantize(codes.data_ptr(), scales.data_ptr(), _ptr(tensor_scale), rows, cols, f,
                                    BLOCK[f], sf, out.data_ptr(), od, _stream(stream))
    _check(st, "fp4_dequantize")
    return out


def fp4_gemm(a_codes: torch.Tensor, a_scales: torch.Tensor, b_codes: torch.Tensor, b_scales: torch.Tensor,
             fmt="mxfp4", a_tensor_scale=None, b_tensor_scale=None, out_dtype="bf16", *, out=None,
             stream=None) -> torch.Tensor:
    """Y[M,N] = alpha * A . B^T on the FP4 tensor cores; scales in the tensor-core ("mma") layout."""
    for t, n in ((a_codes, "a_codes"), (b_codes, "b_codes"), (a_scales, "a_scales"), (b_scales, "b_scales")):
        _need_cuda(t, n)
    f, od = _FMT[fmt], _OUT[out_dtype]
    M, kb = a_codes.shape
    N, kb2 = b_codes.shape
    if kb != kb2:
        raise ValueError("A and B must have the same K")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32 if od == OUT_F32 else torch.bfloat16, device=a_codes.device)
    st = _lib.load().fp4_gemm(a_codes.data_ptr(), a_scales.data_ptr(), _ptr(a_tensor_scale), b_codes.data_ptr(),
                              b_scales.data_ptr(), _ptr(b_tensor_scale), M, N, 2 * kb, f, BLOCK[f],
                              out.data_ptr(), out.stride(0), od, _stream(stream))
    _check(st, "fp4_gemm")
    return out


def fp4_gemm_quantize(a_codes: torch.Tensor, a_scales: torch.Tensor, b_codes: torch.Tensor, b_scales: torch.Tensor,
                      fmt="mxfp4", a_tensor_scale=None, b_tensor_scale=None, out_fmt="mxfp4", rnd="rtn", seed: int = 0,
                      out_tensor_scale: Optional[torch.Tensor] = None, out_sf_layout="mma", *, codes=None, scales=None,
                      stream=None) -> Fp4Quantized:
    """Y = alpha * A . B^T quantized along its rows in the GEMM epilogue (see fp4_gemm_quantize in
    include/fp4.h): the next layer's FP4 operand, Y itself never written."""
    for t, n in ((a_codes, "a_codes"), (b_codes, "b_codes"), (a_scales, "a_scales"), (b_scales, "b_scales")):
        _need_cuda(t, n)
    f, of, r, sf = _FMT[fmt], _FMT[out_fmt], _RND[rnd], _SF[out_sf_layout]
    M, kb = a_codes.shape
    N, kb2 = b_codes.shape
    if kb != kb2:
        raise ValueError("A and B must have the same K")
    if codes is None:
        codes = torch.empty((M, N // 2), dtype=torch.uint8, device=a_codes.device)
    if scales is None:
        nbytes = fp4_scales_bytes(M, N, BLOCK[of], 1, sf)
        shape = (M, N // BLOCK[of]) if sf == SF_ROWMAJOR else (nbytes,)
        scales = torch.empty(shape, dtype=torch.uint8, device=a_codes.device)
    st = _lib.load().fp4_gemm_quantize(
        a_codes.data_ptr(), a_scales.data_ptr(), _ptr(a_tensor_scale), b_codes.data_ptr(), b_scales.data_ptr(),
        _ptr(b_tensor_scale), M, N, 2 * kb, f, BLOCK[f], of, BLOCK[of], r, seed & (2 ** 64 - 1),
        _ptr(out_tensor_scale), codes.data_ptr(), scales.data_ptr(), sf, _stream(stream))
    _check(st, "fp4_gemm_quantize")
    return Fp4Quantized(codes, scales, out_tensor_scale if of == NVFP4 else None)


def fp4_amax(x: torch.Tensor, *, out=None, stream=None) -> torch.Tensor:
    """max |x| of a bf16 matrix as a device fp32 [1]."""
    _bf16_matrix(x)
    if out is None:
        out = torch.empty((1,), dtype=torch.float32, device=x.device)
    _check(_lib.load().fp4_amax(x.data_ptr(), x.shape[0], x.shape[1], x.stride(0), out.data_ptr(),
                                _stream(stream)), "fp4_amax")
    return out


def fp4_nv_tensor_scale(amax: torch.Tensor, *, out=None, stream=None) -> torch.Tensor:
    """NVFP4 tensor scale amax / (6 * 448) (1.0 for amax == 0), computed on the device."""
    _need_cuda(amax, "amax")
    if out is None:
        out = torch.empty((1,), dtype=torch.float32, device=amax.device)
    _check(_lib.load().fp4_nv_tensor_scale(amax.data_ptr(), out.data_ptr(), _stream(stream)),
           "fp4_nv_tensor_scale")
    return out


# ------------------------------------------------------------ 8-bit operators ---
# A small call's time is the host's: the checks below are a comparison each, messages are made where one fails.
_bf16, _f32, _u8 = torch.bfloat16, torch.float32, torch.uint8
_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _elsewhere(fn, x: torch.Tensor, stream, *args, **kwargs):
    """`fn` with its first tensor's device current and, if given, on `stream`: outputs and workspaces are then
    allocated for the stream that uses them."""
    _need_cuda(x, "the first argument")
    if stream is not None and stream.device != x.device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {x.device}")
    with torch.cuda.device(x.device), torch.cuda.stream(stream):
        return fn(x, *args, **kwargs)


def _fits(t: torch.Tensor, dev: int, dtype, shape, name: str) -> torch.Tensor:
    """A contiguous tensor of this dtype and shape on the device."""
    if t.get_device() != dev or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{dev}")
    return t


def _bf16_rows(t: torch.Tensor, dev: int, shape, name: str) -> int:
    """Row stride of a bf16 matrix of this shape (a single row's own stride says nothing)."""
    if t.get_device() != dev or t.dtype is not _bf16 or t.shape != shape or t.stride(1) != 1:
        raise ValueError(f"{name} must be a bf16 tensor of shape {tuple(shape)} with unit column stride on cuda:{dev}")
    return t.stride(0) if shape[0] != 1 else shape[1]


def _codes8(t: torch.Tensor, dev: int, fmt: int, name: str, shape=None) -> int:
    """Row stride of 8-bit codes, bytes or the format's own type (a single row: its length rounded up to 16)."""
    if t.get_device() != dev or t.dtype not in _CODE8[fmt] or t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] != 1) or \
            (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be a matrix of {_CODE8[fmt][1]} codes or bytes" +
                         (f" of shape {tuple(shape)}" if shape is not None else "") + f" with unit column stride on cuda:{dev}")
    rows, cols = t.shape
    return t.stride(0) if rows != 1 else (cols + 15) // 16 * 16


def _scales_shape(rows: int, length: int, sf: int):
    g = (length + FP8_BLOCK - 1) // FP8_BLOCK
    return ((rows + 127) // 128 * 128 * ((g + 3) // 4 * 4),) if sf == SF_MMA else (rows, g)


def _scales8(t: torch.Tensor, dev: int, rows: int, length: int, sf: int, name: str) -> int:
    """Address of checked scale bytes."""
    shape = _scales_shape(rows, length, sf)
    if t.get_device() != dev or t.dtype not in _SCALE8 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous scale bytes of shape {shape} on cuda:{dev}")
    return t.data_ptr()


def _fp8_outputs(x, dev, rows, length, f, sf, codes, scales, name=""):
    """Checked or new codes [rows, length] and scales: (codes, row stride, scales).  New rows that are not whole
    16-byte pieces are padded to 128 bytes: the product reads 128-byte pieces of them, and rows 16 bytes off
    the next line cost it a fifth of its rate."""
    if codes is None:
        if length % 16 == 0:
            pitch, codes = length, x.new_empty((rows, length), dtype=_u8)
        else:
            pitch = (length + 127) // 128 * 128
            codes = x.new_empty((rows, pitch), dtype=_u8)[:, :length]
    else:
        pitch = _codes8(codes, dev, f, "codes" + name, (rows, length))
    if scales is None:
        scales = x.new_empty(_scales_shape(rows, length, sf), dtype=_u8)
    else:
        _scales8(scales, dev, rows, length, sf, "scales" + name)
    return codes, pitch, scales


def fp4_fp8_scales_bytes(rows: int, cols: int, axis: int, sf_layout="rowmajor") -> int:
    """Bytes of 8-bit block scales (128 elements a block) for a [rows, cols] tensor quantized along `axis`;
    0 for an invalid shape."""
    return _lib.load().fp4_fp8_scales_bytes(rows, cols, axis, _SF[sf_layout])


def fp4_fp8_quantize(x: torch.Tensor, fmt="e4m3", axis: int = 1, sf_layout="rowmajor", *, codes=None, scales=None,
                     stream=None) -> Fp8Quantized:
    """bf16 [rows, cols] -> E4M3 or E5M2 codes with one power-of-two scale per 128 elements along `axis` (0: of
    the transpose); see fp4_fp8_quantize in include/fp4.h."""
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _device():
        return _elsewhere(fp4_fp8_quantize, x, stream, fmt, axis, sf_layout, codes=codes, scales=scales)
    _bf16_matrix(x)
    f, sf = _FMT8[fmt], _SF[sf_layout]
    rows, cols = x.shape
    orows, length = (rows, cols) if axis == 1 else (cols, rows)
    codes, pitch, scales = _fp8_outputs(x, dev, orows, length, f, sf, codes, scales)
    _check(_lib.load().fp4_fp8_quantize(x.data_ptr(), rows, cols, x.stride(0) if rows != 1 else cols, f, axis,
                                        codes.data_ptr(), pitch, scales.data_ptr(), sf, _raw_stream(dev)),
           "fp4_fp8_quantize")
    return Fp8Quantized(codes, scales)


def fp4_fp8_quantize_2d(x: torch.Tensor, fmt="e4m3", sf_layout="rowmajor", transposed: bool = True, *, codes=None,
                        scales=None, codes_t=None, scales_t=None, stream=None):
    """One scale per 128 x 128 tile of a bf16 matrix (see fp4_fp8_quantize_2d in include/fp4.h).  Returns
    (W along its rows, W^T along its rows or None) as Fp8Quantized, with the same codes."""
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _device():
        return _elsewhere(fp4_fp8_quantize_2d, x, stream, fmt, sf_layout, transposed, codes=codes, scales=scales,
                          codes_t=codes_t, scales_t=scales_t)
    _bf16_matrix(x)
    f, sf = _FMT8[fmt], _SF[sf_layout]
    rows, cols = x.shape
    codes, pitch, scales = _fp8_outputs(x, dev, rows, cols, f, sf, codes, scales)
    pitch_t = 0
    if transposed:
        codes_t, pitch_t, scales_t = _fp8_outputs(x, dev, cols, rows, f, sf, codes_t, scales_t, "_t")
    elif codes_t is not None or scales_t is not None:
        raise ValueError("codes_t or scales_t is given without transposed")
    _check(_lib.load().fp4_fp8_quantize_2d(x.data_ptr(), rows, cols, x.stride(0) if rows != 1 else cols, f,
                                           codes.data_ptr(), pitch, scales.data_ptr(), _ptr(codes_t), pitch_t,
                                           _ptr(scales_t), sf, _raw_stream(dev)), "fp4_fp8_quantize_2d")
    return Fp8Quantized(codes, scales), (Fp8Quantized(codes_t, scales_t) if transposed else None)


def fp4_fp8_dequantize(codes: torch.Tensor, scales: torch.Tensor, fmt="e4m3", sf_layout="rowmajor", out_dtype="f32", *,
                       out=None, stream=None) -> torch.Tensor:
    """8-bit codes and scales back to fp32 or bf16 [rows, L]."""
    dev = codes.get_device()
    if stream is not None or dev < 0 or dev != _device():
        return _elsewhere(fp4_fp8_dequantize, codes, stream, scales, fmt, sf_layout, out_dtype, out=out)
    f, sf, od = _FMT8[fmt], _SF[sf_layout], _OUT[out_dtype]
    pitch = _codes8(codes, dev, f, "codes")
    rows, cols = codes.shape
    sptr = _scales8(scales, dev, rows, cols, sf, "scales")
    dtype = _f32 if od == OUT_F32 else _bf16
    if out is None:
        out = codes.new_empty((rows, cols), dtype=dtype)
    else:
        _fits(out, dev, dtype, (rows, cols), "out")
    _check(_lib.load().fp4_fp8_dequantize(codes.data_ptr(), pitch, sptr, rows, cols, f, sf, out.data_ptr(), od,
                                          _raw_stream(dev)), "fp4_fp8_dequantize")
    return out


def fp4_fp8_gemm(a_codes: torch.Tensor, a_scales: torch.Tensor, b_codes: torch.Tensor, b_scales: torch.Tensor,
                 a_fmt="e4m3", b_fmt="e4m3", out_dtype="bf16", *, out=None, stream=None) -> torch.Tensor:
    """Y[M, N] = A . B^T of block-scaled 8-bit operands [M, K] and [N, K] on the tensor cores (see fp4_fp8_gemm in
    include/fp4.h); scales in the tensor-core ("mma") layout.  With `out`, its dtype decides."""
    dev = a_codes.get_device()
    if stream is not None or dev < 0 or dev != _device():
        return _elsewhere(fp4_fp8_gemm, a_codes, stream, a_scales, b_codes, b_scales, a_fmt, b_fmt, out_dtype, out=out)
    af, bf = _FMT8[a_fmt], _FMT8[b_fmt]
    lda, ldb = _codes8(a_codes, dev, af, "a_codes"), _codes8(b_codes, dev, bf, "b_codes")
    M, K = a_codes.shape
    N, kb = b_codes.shape
    if kb != K:
        raise ValueError("A and B must have the same K")
    asp, bsp = _scales8(a_scales, dev, M, K, SF_MMA, "a_scales"), _scales8(b_scales, dev, N, K, SF_MMA, "b_scales")
    if out is None:
        od, ldy = _OUT[out_dtype], N
        out = a_codes.new_empty((M, N), dtype=_f32 if od == OUT_F32 else _bf16)
    else:
        od, ldy = out.dtype, out.stride(0) if M != 1 else N
        if od is not _bf16 and od is not _f32 or out.get_device() != dev or out.shape != (M, N) or \
                (out.stride(1) != 1 and N != 1):
            raise ValueError(f"out must be a bf16 or fp32 tensor of shape {(M, N)} with unit column stride on cuda:{dev}")
        od = OUT_BF16 if od is _bf16 else OUT_F32
    _check(_lib.load().fp4_fp8_gemm(a_codes.data_ptr(), lda, asp, b_codes.data_ptr(), ldb, bsp, M, N, K, af, bf,
                                    out.data_ptr(), ldy, od, _raw_stream(dev)), "fp4_fp8_gemm")
    return out


def _norm_weight(weight: torch.Tensor, dev: int, cols: int) -> int:
    if weight.get_device() != dev or weight.dtype is not _bf16 and weight.dtype is not _f32 or \
            weight.shape != (cols,) or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous bf16 or fp32 tensor of shape ({cols},) on cuda:{dev}")
    return OUT_BF16 if weight.dtype is _bf16 else OUT_F32


def fp4_rmsnorm_fp8_quantize(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
                             eps: float = 1e-6, fmt="e4m3", sf_layout="rowmajor", *, codes=None, scales=None,
                             residual_out=None, rstd=None, norm_out=None, stream=None) -> Fp8RmsNorm:
    """h = x + residual (bf16), y = h / sqrt(mean(h^2) + eps) * weight along the rows, y in 8-bit codes and scales,
    in one pass (see fp4_rmsnorm_fp8_quantize in include/fp4.h).  norm_out: a bf16 [rows, cols] tensor that
    receives y as well."""
    dev = x.get_device()
    if stream is not None or dev < 0 or dev != _device():
        return _elsewhere(fp4_rmsnorm_fp8_quantize, x, stream, weight, residual, eps, fmt, sf_layout, codes=codes,
                          scales=scales, residual_out=residual_out, rstd=rstd, norm_out=norm_out)
    _bf16_matrix(x)
    f, sf = _FMT8[fmt], _SF[sf_layout]
    rows, cols = shape = x.shape
    wd = _norm_weight(weight, dev, cols)
    ldr, rptr, hptr, yptr = 0, None, None, None
    if residual is not None:
        ldr, rptr = _bf16_rows(residual, dev, shape, "residual"), residual.data_ptr()
        if residual_out is None:
            residual_out = torch.empty_like(x) if x.is_contiguous() else x.new_empty(shape)
        else:
            _fits(residual_out, dev, _bf16, shape, "residual_out")
        hptr = residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out is given without a residual")
    if rstd is None:
        rstd = x.new_empty((rows,), dtype=_f32)
    else:
        _fits(rstd, dev, _f32, (rows,), "rstd")
    if norm_out is not None:
        yptr = _fits(norm_out, dev, _bf16, shape, "norm_out").data_ptr()
    codes, pitch, scales = _fp8_outputs(x, dev, rows, cols, f, sf, codes, scales)
    _check(_lib.load().fp4_rmsnorm_fp8_quantize(
        x.data_ptr(), x.stride(0) if rows != 1 else cols, rptr, ldr, weight.data_ptr(), wd, rows, cols, eps, f,
        codes.data_ptr(), pitch, scales.data_ptr(), sf, hptr, rstd.data_ptr(), yptr, _raw_stream(dev)),
        "fp4_rmsnorm_fp8_quantize")
    return Fp8RmsNorm(codes, scales, residual_out, rstd)


def fp4_rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                         dresidual: Optional[torch.Tensor] = None, *, dx=None, dweight=None, workspace=None, stream=None):
    """Gradients of y = h * rstd * weight: (dx, the bf16 gradient of h -- of x and of residual alike -- plus
    `dresidual` where given, dweight in fp32).  See fp4_rmsnorm_backward in include/fp4.h."""
    dev = dy.get_device()
    if stream is not None or dev < 0 or dev != _device():
        return _elsewhere(fp4_rmsnorm_backward, dy, stream, h, weight, rstd, dresidual, dx=dx, dweight=dweight,
                          workspace=workspace)
    _bf16_matrix(dy, "dy")
    rows, cols = shape = dy.shape
    ldh, wd = _bf16_rows(h, dev, shape, "h"), _norm_weight(weight, dev, cols)
    _fits(rstd, dev, _f32, (rows,), "rstd")
    lddr, drptr = (0, None) if dresidual is None else (_bf16_rows(dresidual, dev, shape, "dresidual"), dresidual.data_ptr())
    if dx is None:
        dx = torch.empty_like(dy) if dy.is_contiguous() else dy.new_empty(shape)
    else:
        _fits(dx, dev, _bf16, shape, "dx")
    if dweight is None:
        dweight = dy.new_empty((cols,), dtype=_f32)
    else:
        _fits(dweight, dev, _f32, (cols,), "dweight")
    lib = _lib.load()
    if workspace is None:
        # an invalid shape needs 0 bytes: the call below refuses it
        nbytes = lib.fp4_rmsnorm_backward_workspace(rows, cols)
        workspace = dy.new_empty((nbytes or 16,), dtype=_u8)
    else:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
        nbytes = workspace.numel() * workspace.element_size()
    _check(lib.fp4_rmsnorm_backward(
        dy.data_ptr(), dy.stride(0) if rows != 1 else cols, h.data_ptr(), ldh, weight.data_ptr(), wd, rstd.data_ptr(),
        drptr, lddr, rows, cols, dx.data_ptr(), dweight.data_ptr(), workspace.data_ptr(), nbytes, _raw_stream(dev)),
        "fp4_rmsnorm_backward")
    return dx, dweight
