"""What the calls on torch tensors share: streams, dtype codes, argument errors."""
from __future__ import annotations

import torch
from torch.autograd import forward_ad

from . import _native as N

DTYPE_CODES = {torch.float32: N.MOE_DTYPE_F32, torch.bfloat16: N.MOE_DTYPE_BF16, torch.float16: N.MOE_DTYPE_F16,
               torch.int8: N.MOE_DTYPE_S8}


def invalid(what: str, why: str):
    raise ValueError(f"{what}: {why}")


def want(cond: bool, what: str, why: str):
    if not cond:
        invalid(what, why)


def check(status: int, what: str):
    if status != N.MOE_OK:
        raise N.MoeError(status, what)


def vector(t, name, n, what, device, dtype=torch.float32):
    """A 1-D tensor of n values without gaps on the device."""
    if t.dtype is not dtype or t.dim() != 1 or t.shape[0] != n or t.device != device:
        invalid(what, f"{name} must be {dtype} [{n}] on {device}")
    return t if t.is_contiguous() else t.contiguous()


_current = torch._C._cuda_getCurrentRawStream   # the current stream's handle without a Stream object (2 us)


def current_stream(device) -> int:
    return _current(device.index)


def refuse_tangents(what: str, *tensors):
    """Forward-mode derivatives: there are none, and a tangent is not dropped without a word."""
    if forward_ad._current_level >= 0:
        for t in tensors:
            if t is not None and forward_ad.unpack_dual(t).tangent is not None:
                invalid(what, "has no forward-mode derivative, and an input has a tangent")


def refuse_gradients(what: str, *tensors):
    """The call has no gradient: an input that records one would lose it without a word."""
    if forward_ad._current_level >= 0:
        refuse_tangents(what, *tensors)
    for t in tensors:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            invalid(what, "has no gradient, and an input requires one: detach it, or call under torch.no_grad()")


_device = torch._C._cuda_getDevice   # the current device's index, likewise


def elsewhere(t) -> bool:
    """Whether the tensor is on another device than the current one, on which a kernel would start."""
    index = t.get_device()   # -1: no CUDA tensor
    return index >= 0 and index != _device()


def run_on(stream, fn, first, *args):
    """fn(first, *args) on the device of the tensor `first`, with `stream` as the current one, so that what it
    allocates belongs to that stream; None: the device's own current stream. The allocator learns that the
    inputs are in use on `stream`, and the outputs on the caller's: a tensor freed after the call is not handed
    out again before both are done with it. (What comes first on which stream stays the caller's business.)"""
    if stream is None:
        with torch.cuda.device(first.device):
            return fn(first, *args)
    if first.is_cuda and stream.device != first.device:
        invalid(fn.__name__, f"the stream is on {stream.device}, the tensors are on {first.device}")
    caller = torch.cuda.current_stream(first.device) if first.is_cuda else stream
    with torch.cuda.stream(stream):
        out = fn(first, *args)
    if caller != stream:
        for t in (first, *args):
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)
        for t in out if isinstance(out, tuple) else (out,):
            t.record_stream(caller)
    return out
