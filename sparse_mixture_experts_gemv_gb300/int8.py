"""Projections and SwiGLU experts in 8-bit integers (moe_quant_* in the C ABI), with a
scale for each token and channel. Argument checks and marshalling only."""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _native as N
from ._tensors import DTYPE_CODES, check, counts32, current_stream, elsewhere, invalid, refuse_gradients, run_on, vector, want


@functools.lru_cache(maxsize=256)
def _matmul_workspace(T, n, K, code):
    b = ctypes.c_int64()
    check(N.load().moe_quant_matmul_workspace(T, n, K, code, ctypes.byref(b)), "moe_quant_matmul_workspace")
    return b.value


@functools.lru_cache(maxsize=256)
def _experts_config(E, k, H, I, T):
    cfg = N.moe_int8_experts_config_t(E, k, H, I)
    b = ctypes.c_int64()
    check(N.load().moe_quant_experts_workspace(ctypes.byref(cfg), T, ctypes.byref(b)), "moe_quant_experts_workspace")
    return ctypes.byref(cfg), b.value


def _rows(t, K, what, name):
    """A matrix whose rows the kernels can read (16-byte addresses and row strides), its address and row stride."""
    size, ptr = t.element_size(), t.data_ptr()
    stride, inner = t.stride()
    if inner != 1 or stride < K or (ptr | stride * size) & 15:
        t = t.clone(memory_format=torch.contiguous_format)
        ptr, stride = t.data_ptr(), K
        want(K * size % 16 == 0, what, f"the rows of {name} must be a multiple of 16 bytes long")
    return t, ptr, stride


def int8_matmul(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, x_scale: torch.Tensor = None,
                out_dtype: torch.dtype = None, stream: torch.cuda.Stream = None) -> torch.Tensor:
    """out[t, n] = (sum_k q[t, k] w[n, k]) x_scale[t] w_scale[n].

    w: int8 [N, K], w_scale: fp32 [N]. x [T, K]: int8 with x_scale fp32 [T], or bf16, fp16 or
    fp32 without: each row is then quantized by the call, its scale being its largest magnitude
    times fp32(1/127) (what amax / 127 is for a tensor on the GPU; the rounded quotient differs
    by a step in some rows), to the nearest whole number (a row with an infinity or a NaN gives
    NaN). K is a multiple of 16. Rows may be apart (any stride(0)); rows off 16-byte boundaries are copied first.
    out_dtype: bf16, fp16 or fp32; by default x's, and bf16 for int8 x. There is no gradient:
    inputs that require one are refused while gradients are recorded.
    """
    if stream is not None or elsewhere(x):
        return run_on(stream, int8_matmul, x, w, w_scale, x_scale, out_dtype)
    what = "int8_matmul"
    refuse_gradients(what, x, w_scale, x_scale)
    code = DTYPE_CODES.get(x.dtype)
    if code is None or not x.is_cuda or x.dim() != 2:
        invalid(what, "x must be a CUDA tensor [T, K] of int8, bf16, fp16 or fp32")
    T, K = x.shape
    dev = x.device
    if w.dtype is not torch.int8 or w.dim() != 2 or w.shape[1] != K or w.device != dev:
        invalid(what, f"w must be int8 [N, {K}] on {dev}")
    n = w.shape[0]
    counts32(what, T, n, K)
    w_scale = vector(w_scale, "w_scale", n, what, dev)
    quantized = code == N.MOE_DTYPE_S8
    if quantized != (x_scale is not None):
        invalid(what, "x_scale goes with int8 x, and with no other")
    if quantized:
        x_scale = vector(x_scale, "x_scale", T, what, dev)
    if out_dtype is None:
        out_dtype = torch.bfloat16 if quantized else x.dtype
    out_code = DTYPE_CODES.get(out_dtype)
    if out_code is None or out_code == N.MOE_DTYPE_S8:
        invalid(what, "out_dtype must be bf16, fp16 or fp32")
    out = torch.empty((T, n), dtype=out_dtype, device=dev)
    if T == 0 or n == 0:
        return out
    x, x_ptr, x_stride = _rows(x, K, what, "x")
    w, w_ptr, w_stride = _rows(w, K, what, "w")
    need = _matmul_workspace(T, n, K, code)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    status = N.load().moe_quant_matmul(x_ptr, code, x_stride, None if x_scale is None else x_scale.data_ptr(), w_ptr,
                                       w_stride, w_scale.data_ptr(), out.data_ptr(), out_code, T, n, K,
                                       None if ws is None else ws.data_ptr(), need, current_stream(dev))
    if status:
        check(status, "moe_quant_matmul")
    return out


def int8_experts(x: torch.Tensor, idx: torch.Tensor, weights: torch.Tensor, gate_up: torch.Tensor,
                 gate_up_scale: torch.Tensor, down: torch.Tensor, down_scale: torch.Tensor,
                 stream: torch.cuda.Stream = None) -> torch.Tensor:
    """out[t] = sum_j weights[t, j] * expert[idx[t, j]](x[t]) with SwiGLU experts in int8.

    x: bf16 or fp16 [T, H]. idx int32 and weights fp32 [T, k] as route_experts gives them; a
    choice outside [0, E) contributes nothing. gate_up: int8 [E, 2I, H], gate rows before up
    rows, gate_up_scale fp32 [E, 2I]; down: int8 [E, H, I], down_scale fp32 [E, H];
    these four without gaps and on 16-byte boundaries. H and I are multiples of 16. x and the
    SwiGLU outputs are quantized for each token as in int8_matmul. Returns [T, H] in x's type.
    There is no gradient: inputs that require one, weights with a router's graph among them,
    are refused while gradients are recorded.
    """
    if stream is not None or elsewhere(x):
        return run_on(stream, int8_experts, x, idx, weights, gate_up, gate_up_scale, down, down_scale)
    what = "int8_experts"
    refuse_gradients(what, x, weights, gate_up_scale, down_scale)
    if not x.is_cuda or x.dim() != 2 or (x.dtype is not torch.bfloat16 and x.dtype is not torch.float16):
        invalid(what, "x must be a CUDA tensor [T, H] of bf16 or fp16")
    T, H = x.shape
    dev = x.device
    if idx.dim() != 2 or idx.shape[0] != T or idx.dtype is not torch.int32 or idx.device != dev:
        invalid(what, f"idx must be int32 [{T}, k] on {dev}")
    k = idx.shape[1]
    if weights.shape != idx.shape or weights.dtype is not torch.float32 or weights.device != dev:
        invalid(what, f"weights must be fp32 [{T}, {k}] on {dev}")
    if gate_up.dim() != 3 or gate_up.shape[2] != H or gate_up.shape[1] % 2 or gate_up.dtype is not torch.int8:
        invalid(what, f"gate_up must be int8 [E, 2I, {H}]")
    E, I = gate_up.shape[0], gate_up.shape[1] // 2
    if E == 0 or I == 0:
        invalid(what, "there must be an expert and an intermediate feature")
    counts32(what, T, k, E, H, I)
    if down.shape != (E, H, I) or down.dtype is not torch.int8:
        invalid(what, f"down must be int8 [{E}, {H}, {I}]")
    if gate_up_scale.shape != (E, 2 * I) or gate_up_scale.dtype is not torch.float32:
        invalid(what, f"gate_up_scale must be fp32 [{E}, {2 * I}]")
    if down_scale.shape != (E, H) or down_scale.dtype is not torch.float32:
        invalid(what, f"down_scale must be fp32 [{E}, {H}]")
    w = N.moe_int8_experts_weights_t(gate_up.data_ptr(), gate_up_scale.data_ptr(), down.data_ptr(),
                                     down_scale.data_ptr())
    if (w.gate_up_dev | w.gate_up_scale_dev | w.down_dev | w.down_scale_dev) & 15 or not (
            gate_up.is_contiguous() and gate_up_scale.is_contiguous() and down.is_contiguous() and
            down_scale.is_contiguous()) or not (
            gate_up.device == gate_up_scale.device == down.device == down_scale.device == dev):
        invalid(what, f"the weights and their scales must be on {dev}, without gaps and on 16-byte boundaries")
    x, idx, weights = x.contiguous(), idx.contiguous(), weights.contiguous()
    if x.data_ptr() & 15:
        x = x.clone()
    out = torch.empty((T, H), dtype=x.dtype, device=dev)
    if T == 0:
        return out
    cfg, need = _experts_config(E, k, H, I, T)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    check(N.load().moe_quant_experts(cfg, ctypes.byref(w), x.data_ptr(), DTYPE_CODES[x.dtype], idx.data_ptr(),
                                    weights.data_ptr(), out.data_ptr(), T, ws.data_ptr(), need,
                                    current_stream(dev)), "moe_quant_experts")
    return out


def int8_sync_status(stream: torch.cuda.Stream = None) -> int:
    """Waits for the stream; MOE_OK, or MOE_ERR_TIMEOUT if a product's bounded wait ran out on its device since the last call."""
    stream = stream or torch.cuda.current_stream()
    with torch.cuda.device(stream.device):
        return N.load().moe_quant_sync_status(stream.cuda_stream)
