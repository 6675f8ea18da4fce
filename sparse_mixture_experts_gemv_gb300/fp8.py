"""Rows and products in 8-bit floating point (E4M3) with a scale for each block of 128
(moe_block_* in the C ABI). Argument checks and marshalling only."""
from __future__ import annotations

import torch

from . import _native as N
from ._tensors import check, counts32, current_stream, elsewhere, invalid, refuse_gradients, rows16, run_on

FLOAT_CODES = {torch.float32: N.MOE_DTYPE_F32, torch.bfloat16: N.MOE_DTYPE_BF16, torch.float16: N.MOE_DTYPE_F16}
ROW_CODES = {**FLOAT_CODES, torch.float8_e4m3fn: N.MOE_DTYPE_E4M3}
BLOCK = 128


def _blocks(n):
    return -(-n // BLOCK)


def _pad256(n):
    return -(-n // 256) * 256


def _row_scales(scale, rows, K, what, device):
    if scale.shape != (rows, _blocks(K)) or scale.dtype is not torch.float32 or scale.device != device:
        invalid(what, f"x_scale must be fp32 [{rows}, {_blocks(K)}] on {device}")
    return scale.contiguous()


def fp8_quantize(x: torch.Tensor, swiglu: bool = False, stream: torch.cuda.Stream = None):
    """Rows to E4M3 with a scale for each block of 128 values: (q float8_e4m3fn [T, K], scale fp32 [T, ceil(K / 128)]).

    x: fp32, bf16 or fp16 [T, K], K a multiple of 16, rows any distance apart (rows off 16-byte boundaries are
    copied first). swiglu: x is [T, 2K], gate before up, and g / (1 + e^-g) * u is quantized. A block's
    scale is its largest magnitude times fp32(1/448), which is what amax / 448 is for a tensor on
    the GPU, or 1 where that is 0; the quotient by it is rounded to fp32, and that to the nearest
    E4M3 value. A block with an infinity or a NaN has the scale NaN. There is no gradient: inputs
    that require one are refused while gradients are recorded.
    """
    if stream is not None or elsewhere(x):
        return run_on(stream, fp8_quantize, x, swiglu)
    what = "fp8_quantize"
    refuse_gradients(what, x)
    code = FLOAT_CODES.get(x.dtype)
    if code is None or not x.is_cuda or x.dim() != 2 or x.shape[1] == 0 or (swiglu and x.shape[1] % 2):
        invalid(what, "x must be a CUDA tensor [T, K] (swiglu: [T, 2K]) of fp32, bf16 or fp16")
    T, width = x.shape
    K = width // 2 if swiglu else width
    counts32(what, T, K)
    q = torch.empty((T, K), dtype=torch.float8_e4m3fn, device=x.device)
    scale = torch.empty((T, _blocks(K)), dtype=torch.float32, device=x.device)
    x, ptr, stride = rows16(x, width, what, "x")
    status = N.load().moe_block_quantize(ptr, code, stride, 1 if swiglu else 0, T, K, q.data_ptr(), scale.data_ptr(),
                                         current_stream(x.device))
    if status:
        check(status, "moe_block_quantize")
    return q, scale


def _product(what, x, offsets, w, w_scale, x_scale, out_dtype):
    refuse_gradients(what, x, w, w_scale, x_scale)
    code = ROW_CODES.get(x.dtype)
    if code is None or not x.is_cuda or x.dim() != 2:
        invalid(what, "x must be a CUDA tensor [rows, K] of float8_e4m3fn, bf16, fp16 or fp32")
    M, K = x.shape
    dev = x.device
    lead = w.shape[:-2]
    if w.dtype is not torch.float8_e4m3fn or w.dim() != (2 if offsets is None else 3) or w.shape[-1] != K or w.device != dev:
        invalid(what, f"w must be float8_e4m3fn [{'N' if offsets is None else 'E, N'}, {K}] on {dev}")
    n = w.shape[-2]
    counts32(what, M, n, K, *lead)
    if w_scale.shape != (*lead, _blocks(n), _blocks(K)) or w_scale.dtype is not torch.float32 or w_scale.device != dev:
        invalid(what, f"w_scale must be fp32 {[*lead, _blocks(n), _blocks(K)]} on {dev}")
    w_scale = w_scale.contiguous()
    quantized = code == N.MOE_DTYPE_E4M3
    if quantized != (x_scale is not None):
        invalid(what, "x_scale goes with float8_e4m3fn x, and with no other")
    if quantized:
        x_scale = _row_scales(x_scale, M, K, what, dev)
    if out_dtype is None:
        out_dtype = torch.bfloat16 if quantized else x.dtype
    out_code = FLOAT_CODES.get(out_dtype)
    if out_code is None:
        invalid(what, "out_dtype must be bf16, fp16 or fp32")
    if offsets is not None:
        if lead[0] == 0 or offsets.dim() != 1 or offsets.shape[0] != lead[0] + 1 or offsets.dtype is not torch.int32 or (
                offsets.device != dev):
            invalid(what, f"offsets must be int32 [{lead[0] + 1}] on {dev}, of at least one expert")
        if not w.is_contiguous() or w.data_ptr() & 15:
            invalid(what, "w must be without gaps and on a 16-byte boundary")
        offsets = offsets.contiguous()
    out = torch.empty((M, n), dtype=out_dtype, device=dev)
    if M == 0 or n == 0:
        return out
    if K % 16 or K == 0:
        invalid(what, "K must be a multiple of 16")
    x, x_ptr, x_stride = rows16(x, K, what, "x")
    # few values are quantized inside the product
    need = 0 if quantized or (M <= 16 and K <= 4096 and M * K <= 20480) else _pad256(M * K) + _pad256(M * _blocks(K) * 4)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    ws_ptr = None if ws is None else ws.data_ptr()
    scale_ptr = None if x_scale is None else x_scale.data_ptr()
    if offsets is None:
        w, w_ptr, w_stride = rows16(w, K, what, "w")
        status = N.load().moe_block_matmul(x_ptr, code, x_stride, scale_ptr, w_ptr, w_stride, w_scale.data_ptr(),
                                           out.data_ptr(), out_code, M, n, K, ws_ptr, need, current_stream(dev))
    else:
        status = N.load().moe_block_grouped_matmul(x_ptr, code, x_stride, scale_ptr, offsets.data_ptr(), w.data_ptr(),
                                                   w_scale.data_ptr(), out.data_ptr(), out_code, M, lead[0], n, K,
                                                   ws_ptr, need, current_stream(dev))
    if status:
        check(status, what)
    return out


def fp8_matmul(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, x_scale: torch.Tensor = None,
               out_dtype: torch.dtype = None, stream: torch.cuda.Stream = None) -> torch.Tensor:
    """out[t, n] = sum_b x_scale[t, b] w_scale[n // 128, b] (sum over block b of x[t, k] w[n, k]).

    w: float8_e4m3fn [N, K], w_scale: fp32 [ceil(N / 128), ceil(K / 128)], a scale for each 128 x 128
    of w; the product of a block's two scales is held in 32 bits. x [T, K]: float8_e4m3fn with x_scale fp32 [T, ceil(K / 128)], or bf16, fp16 or fp32 without: it
    is then quantized by the call as fp8_quantize does. K is a multiple of 16. Rows may be apart (any
    stride(0)); rows off 16-byte boundaries are copied first. out_dtype: bf16, fp16 or fp32; by
    default x's, and bf16 for float8_e4m3fn x. There is no gradient: inputs that require one are refused
    while gradients are recorded.
    """
    if stream is not None or elsewhere(x):
        return run_on(stream, fp8_matmul, x, w, w_scale, x_scale, out_dtype)
    return _product("fp8_matmul", x, None, w, w_scale, x_scale, out_dtype)


def fp8_grouped_matmul(x: torch.Tensor, offsets: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor,
                       x_scale: torch.Tensor = None, out_dtype: torch.dtype = None,
                       stream: torch.cuda.Stream = None) -> torch.Tensor:
    """fp8_matmul of rows in the order of their experts: x[offsets[e]:offsets[e + 1]] is multiplied with w[e].

    x [M, K] and x_scale as there; offsets: int32 [E + 1], as dispatch_tokens gives them; w:
    float8_e4m3fn [E, N, K] without gaps and on a 16-byte boundary, w_scale: fp32 [E, ceil(N / 128),
    ceil(K / 128)]. Rows of no expert (before offsets[0], behind offsets[E]) give rows of zeros.
    Returns [M, N]. There is no gradient, as there.
    """
    if stream is not None or elsewhere(x):
        return run_on(stream, fp8_grouped_matmul, x, offsets, w, w_scale, x_scale, out_dtype)
    if offsets is None:
        invalid("fp8_grouped_matmul", "offsets must be int32 [E + 1]")
    return _product("fp8_grouped_matmul", x, offsets, w, w_scale, x_scale, out_dtype)


def fp8_sync_status(stream: torch.cuda.Stream = None) -> int:
    """Waits for the stream; MOE_OK, or MOE_ERR_TIMEOUT if a product's bounded wait ran out on its device since the last call."""
    stream = stream or torch.cuda.current_stream()
    with torch.cuda.device(stream.device):
        return N.load().moe_block_sync_status(stream.cuda_stream)
