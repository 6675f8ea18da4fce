"""Tokens in the order of their experts and back (moe_dispatch_tokens and
moe_combine_tokens in the C ABI), and the gradients of both. Argument checks and
marshalling only."""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _native as N
from ._tensors import check, counts32, current_stream, elsewhere, gradient, invalid, refuse_gradients, refuse_tangents, run_on

FLOAT_CODES = {torch.float32: N.MOE_DTYPE_F32, torch.bfloat16: N.MOE_DTYPE_BF16, torch.float16: N.MOE_DTYPE_F16}
ROW_TYPES = {torch.float32, torch.bfloat16, torch.float16, torch.float8_e4m3fn, torch.int8, torch.uint8}


def _matrix(t, what, name):
    """A CUDA matrix of fp32, bf16 or fp16: itself or a copy whose rows have no gaps inside, its type's code and row
    stride."""
    code = FLOAT_CODES.get(t.dtype)
    if code is None or not t.is_cuda or t.dim() != 2 or t.shape[1] == 0:
        invalid(what, f"{name} must be a CUDA tensor [rows, H] of fp32, bf16 or fp16")
    rows, H = t.shape
    stride, inner = t.stride()
    if (inner != 1 and H > 1) or (rows > 1 and stride < H):
        t, stride = t.contiguous(), H
    return t, code, stride if rows > 1 else H   # one row has no next one: its stride may be anything


def _pos(pos, rows, what, device):
    if pos.dim() != 2 or pos.dtype is not torch.int32 or pos.device != device or pos.numel() != rows or (
            rows == 0 and pos.shape[1] == 0):
        invalid(what, f"pos must be int32 [T, k] on {device}, with a row for each choice ({rows})")
    return pos.contiguous()


def _weights(weights, pos, what):
    if weights is None:
        return None
    if weights.shape != pos.shape or weights.dtype is not torch.float32 or weights.device != pos.device:
        invalid(what, f"weights must be fp32 {list(pos.shape)} on {pos.device}")
    return weights.contiguous()


def _ptr(t):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=256)
def _workspace(device, T, k, E):
    b = ctypes.c_int64()
    check(N.load().moe_dispatch_tokens_workspace(T, k, E, ctypes.byref(b)), "moe_dispatch_tokens")
    return b.value


def _dispatch(x, idx, num_experts, x_scale):
    what = "dispatch_tokens"
    if x.dtype not in ROW_TYPES or not x.is_cuda or x.dim() != 2 or x.shape[1] == 0:
        invalid(what, "x must be a CUDA tensor [T, H] of fp32, bf16, fp16 or 8 bits")
    T, H = x.shape
    dev = x.device
    if idx.dim() != 2 or idx.shape[0] != T or idx.shape[1] == 0 or idx.dtype is not torch.int32 or idx.device != dev:
        invalid(what, f"idx must be int32 [{T}, k] on {dev}")
    if isinstance(num_experts, torch.Tensor) or not 0 < num_experts < 2 ** 31:
        invalid(what, f"num_experts must be a plain number above 0, not {num_experts}")
    k, size = idx.shape[1], x.element_size()
    stride, inner = x.stride()
    if (inner != 1 and H > 1) or (T > 1 and stride < H):
        x, stride = x.contiguous(), H
    scales = 0
    if x_scale is not None:
        if x_scale.dim() != 2 or x_scale.shape[0] != T or x_scale.dtype is not torch.float32 or x_scale.device != dev:
            invalid(what, f"x_scale must be fp32 [{T}, n] on {dev}")
        x_scale, scales = x_scale.contiguous(), x_scale.shape[1]
        if scales == 0:
            invalid(what, "x_scale must have a scale for each row")
    counts32(what, T, k, scales)
    need = _workspace(dev.index, T, k, num_experts)
    idx = idx.contiguous()
    rows = torch.empty((T * k, H), dtype=x.dtype, device=dev)
    row_scale = torch.empty((T * k, scales), dtype=torch.float32, device=dev) if scales else None
    offsets = torch.empty(num_experts + 1, dtype=torch.int32, device=dev)
    pos = torch.empty((T, k), dtype=torch.int32, device=dev)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    status = N.load().moe_dispatch_tokens(x.data_ptr(), H * size, (stride if T > 1 else H) * size, _ptr(x_scale), scales,
                                          idx.data_ptr(), T, k, num_experts, rows.data_ptr(), _ptr(row_scale),
                                          offsets.data_ptr(), pos.data_ptr(), _ptr(ws), need, current_stream(dev))
    if status:
        check(status, "moe_dispatch_tokens")
    return (rows, offsets, pos) if row_scale is None else (rows, row_scale, offsets, pos)


def _sum(y, pos, weights, what):
    y, code, stride = _matrix(y, what, "y" if weights is not None else "the rows")
    pos = _pos(pos, y.shape[0], what, y.device)
    weights = _weights(weights, pos, what)
    T, k = pos.shape
    H = y.shape[1]
    counts32(what, T, k, H)
    out = torch.empty((T, H), dtype=y.dtype, device=y.device)
    if T == 0:
        return out
    status = N.load().moe_combine_tokens(y.data_ptr(), code, stride, pos.data_ptr(), _ptr(weights), T, k, H,
                                         out.data_ptr(), current_stream(y.device))
    if status:
        check(status, "moe_combine_tokens")
    return out


def _dispatch_backward(d_rows, pos):
    return _sum(d_rows, pos, None, "dispatch_tokens_backward")


def _combine(y, weights, pos):
    return _sum(y, pos, weights, "combine_tokens")


def _combine_gradients(d_out, y, weights, pos, want_y, want_weights):
    what = "combine_tokens_backward"
    y, code, stride = _matrix(y, what, "y")
    pos = _pos(pos, y.shape[0], what, y.device)
    weights = _weights(weights, pos, what)
    T, k = pos.shape
    H, dev = y.shape[1], y.device
    counts32(what, T, k, H)
    if d_out.shape != (T, H) or d_out.dtype is not y.dtype or d_out.device != dev:
        invalid(what, f"d_out must be {y.dtype} [{T}, {H}] on {dev}")
    d_out, _, d_stride = _matrix(d_out, what, "d_out")
    d_y = torch.empty((T * k, H), dtype=y.dtype, device=dev) if want_y else None
    d_weights = torch.empty((T, k), dtype=torch.float32, device=dev) if want_weights else None
    if T == 0:
        return d_y, d_weights
    status = N.load().moe_combine_tokens_backward(d_out.data_ptr(), d_stride, y.data_ptr(), code, stride, pos.data_ptr(),
                                                  _ptr(weights), T, k, H, _ptr(d_y), _ptr(d_weights),
                                                  current_stream(dev))
    if status:
        check(status, "moe_combine_tokens_backward")
    return d_y, d_weights


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, idx, num_experts):
        rows, offsets, pos = _dispatch(x, idx, num_experts, None)
        ctx.save_for_backward(pos)
        ctx.mark_non_differentiable(offsets, pos)
        return rows, offsets, pos

    @staticmethod
    def backward(ctx, d_rows, *_):
        return dispatch_tokens_backward(d_rows, *ctx.saved_tensors), None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, pos):
        ctx.save_for_backward(y, weights, pos)
        return _combine(y, weights, pos)

    @staticmethod
    def backward(ctx, d_out):
        y, weights, pos = ctx.saved_tensors
        d_y, d_weights = gradient("combine_tokens", _combine_gradients, (d_out, y, weights), pos,
                                  *ctx.needs_input_grad[:2])
        return d_y, d_weights, None


def dispatch_tokens(x: torch.Tensor, idx: torch.Tensor, num_experts: int, x_scale: torch.Tensor = None,
                    stream: torch.cuda.Stream = None):
    """Copies each token's row to the places of its k choices, sorted by expert.

    x [T, H]: fp32, bf16, fp16 or 8 bits (E4M3, int8, uint8), rows any distance apart; idx: int32 [T, k] as
    route_experts gives it. Returns (rows [T k, H], offsets int32 [num_experts + 1], pos int32
    [T, k]): rows[pos[t, j]] is x[t], expert e has rows[offsets[e]:offsets[e + 1]], in the order
    of the choices. A choice outside [0, num_experts) has a row of zeros behind the last expert's,
    and pos is ~row, below 0. With x_scale (fp32 [T, n], the scales of quantized rows) the
    result is (rows, row_scale [T k, n], offsets, pos).

    rows of fp32, bf16 or fp16 (without x_scale) are differentiable with respect to x, once; idx has no gradient.
    """
    if stream is not None or elsewhere(x):
        return run_on(stream, dispatch_tokens, x, idx, num_experts, x_scale)
    refuse_tangents("dispatch_tokens", x, x_scale)
    if x_scale is not None or x.dtype not in FLOAT_CODES:
        refuse_gradients("dispatch_tokens of quantized rows", x, x_scale)
    elif x.requires_grad and torch.is_grad_enabled():
        return _Dispatch.apply(x, idx, num_experts)
    return _dispatch(x, idx, num_experts, x_scale)


def dispatch_tokens_backward(d_rows: torch.Tensor, pos: torch.Tensor, stream: torch.cuda.Stream = None):
    """d_x [T, H] from d_rows [T k, H] and the pos of dispatch_tokens: each token's sum over its choices, in 32
    bits, rounded once. It has no derivative itself, and refuses one when it is asked for."""
    if stream is not None or elsewhere(d_rows):
        return run_on(stream, dispatch_tokens_backward, d_rows, pos)
    refuse_tangents("dispatch_tokens_backward", d_rows)
    return gradient("dispatch_tokens", _dispatch_backward, (d_rows,), pos)


def combine_tokens(y: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor, stream: torch.cuda.Stream = None):
    """out[t] = sum_j weights[t, j] * y[pos[t, j]], added up in 32 bits and rounded once.

    y [T k, H]: fp32, bf16 or fp16, the experts' results in the order of dispatch_tokens' rows,
    whose pos int32 [T, k] this is; weights: fp32 [T, k]. A choice of no expert (pos below 0) adds
    nothing. Returns [T, H] in y's type, differentiable with respect to y and weights, once.
    """
    if stream is not None or elsewhere(y):
        return run_on(stream, combine_tokens, y, pos, weights)
    refuse_tangents("combine_tokens", y, weights)
    if weights is None:
        invalid("combine_tokens", "weights must be fp32 [T, k]")
    if torch.is_grad_enabled() and (y.requires_grad or weights.requires_grad):
        return _Combine.apply(y, weights, pos)
    return _combine(y, weights, pos)


def combine_tokens_backward(d_out: torch.Tensor, y: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor,
                            stream: torch.cuda.Stream = None):
    """(d_y [T k, H] in y's type, d_weights fp32 [T, k]) from d_out [T, H] in y's type and what combine_tokens took:
    the row of a choice of no expert is zeros in d_y, and its d_weights 0. They have no derivative
    themselves, and refuse one when it is asked for."""
    if stream is not None or elsewhere(d_out):
        return run_on(stream, combine_tokens_backward, d_out, y, pos, weights)
    refuse_tangents("combine_tokens_backward", d_out, y, weights)
    if weights is None:
        invalid("combine_tokens_backward", "weights must be fp32 [T, k]")
    return gradient("combine_tokens", _combine_gradients, (d_out, y, weights), pos, True, True)
