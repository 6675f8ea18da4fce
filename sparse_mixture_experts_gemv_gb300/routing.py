"""Routing to experts from given logits (moe_route_experts in the C ABI): softmax or
sigmoid scores, a bias that only chooses, groups of experts, top-k, renormalised
weights, and the gradient of the logits. Argument checks and marshalling only."""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _native as N
from ._tensors import DTYPE_CODES, check, counts32, current_stream, elsewhere, invalid, refuse_tangents, run_on, vector, want

LOGIT_CODES = {t: c for t, c in DTYPE_CODES.items() if t is not torch.int8}
SCORES = {"softmax": N.MOE_SCORE_SOFTMAX, "sigmoid": N.MOE_SCORE_SIGMOID}


@functools.lru_cache(maxsize=256)
def _config(E, k, score, groups, top_groups, group_top, renormalise, scale):
    if score not in SCORES:
        invalid("route_experts", f"score must be one of {sorted(SCORES)}")
    # kept by their values: a tensor, which would be kept by its identity, can change
    if any(isinstance(v, torch.Tensor) for v in (k, groups, top_groups, group_top, renormalise, scale)):
        invalid("route_experts", "k, groups, top_groups, group_top, renormalise and scale are plain values, not tensors")
    for n in (k, groups, top_groups, group_top):
        if not 0 <= n < 2 ** 31:
            invalid("route_experts", f"k, groups, top_groups and group_top must be numbers of 31 bits, not {n}")
    return ctypes.byref(N.moe_route_config_t(E, k, SCORES[score], groups, top_groups, group_top,
                                             1 if renormalise else 0, scale))


def _logits(what, logits):
    """The logits with their dtype's code, shape and row stride, copied where rows have gaps inside."""
    code = LOGIT_CODES.get(logits.dtype)
    if code is None or not logits.is_cuda or logits.dim() != 2:
        invalid(what, "logits must be a CUDA tensor [T, E] of fp32, bf16 or fp16")
    T, E = logits.shape
    counts32(what, T, E)
    stride, inner = logits.stride()
    if inner != 1 or stride < E:
        logits, stride = logits.contiguous(), E
    return logits, code, T, E, stride if T > 1 else E   # one row has no next one: its stride may be anything


def _forward(logits, k, score, bias, groups, top_groups, group_top, renormalise, scale):
    logits, code, T, E, stride = _logits("route_experts", logits)
    dev = logits.device
    if bias is not None:
        bias = vector(bias, "bias", E, "route_experts", dev)
    cfg = _config(E, k, score, groups, top_groups, group_top, renormalise, scale)
    idx = torch.empty((T, k), dtype=torch.int32, device=dev)
    weights = torch.empty((T, k), dtype=torch.float32, device=dev)
    status = N.load().moe_route_experts(cfg, logits.data_ptr(), code, stride,
                                        None if bias is None else bias.data_ptr(), T, idx.data_ptr(),
                                        weights.data_ptr(), current_stream(dev))
    if status:
        check(status, "moe_route_experts")
    return idx, weights


def _backward(d_weights, logits, idx, score, renormalise, scale):
    what = "route_experts_backward"
    logits, code, T, E, stride = _logits(what, logits)
    dev = logits.device
    want(idx.dim() == 2 and idx.shape[0] == T and idx.dtype is torch.int32 and idx.device == dev, what,
         "idx must be int32 [T, k] on the logits' device")
    k = idx.shape[1]
    want(d_weights.shape == idx.shape and d_weights.dtype is torch.float32 and d_weights.device == dev, what,
         "d_weights must be fp32 [T, k] on the logits' device")
    idx, d_weights = idx.contiguous(), d_weights.contiguous()
    d_logits = torch.empty((T, E), dtype=logits.dtype, device=dev)
    check(N.load().moe_route_experts_backward(_config(E, k, score, 1, 1, 1, renormalise, scale), logits.data_ptr(),
                                              code, stride,
                                              idx.data_ptr(), d_weights.data_ptr(), T, d_logits.data_ptr(),
                                              current_stream(dev)), "moe_route_experts_backward")
    return d_logits


class _RouteExperts(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, score, bias, groups, top_groups, group_top, renormalise, scale):
        idx, weights = _forward(logits, k, score, bias, groups, top_groups, group_top, renormalise, scale)
        ctx.save_for_backward(logits, idx)
        ctx.how = (score, renormalise, scale)
        ctx.mark_non_differentiable(idx)
        return idx, weights

    @staticmethod
    def backward(ctx, _, d_weights):
        logits, idx = ctx.saved_tensors
        return (route_experts_backward(d_weights, logits, idx, *ctx.how),) + (None,) * 8


class _RouteGradient(torch.autograd.Function):
    """The gradient as a step of a recorded graph: it has no derivative of its own, and says so when asked for one."""

    @staticmethod
    def forward(ctx, *args):
        return _backward(*args)

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("route_experts has no second derivative")


def route_experts(logits: torch.Tensor, k: int, score: str = "softmax", bias: torch.Tensor = None, groups: int = 1,
                  top_groups: int = None, group_top: int = 2, renormalise: bool = True, scale: float = 1.0,
                  stream: torch.cuda.Stream = None):
    """Chooses k experts for each row of logits [T, E] (fp32, bf16 or fp16).

    score: "softmax" or "sigmoid". bias: fp32 [E], added to the scores for the choice alone
    (a bias for balance; it has no gradient). groups > 1: consecutive experts form groups; the top_groups groups
    whose group_top (1 or 2) largest keys add up to most stay. The weights are the scores
    without the bias, divided by their sum if renormalise, times scale. Equal keys go by the
    lower index; a logit of -inf or NaN turns its expert off for the row. A bias of
    -inf or NaN ranks its expert below all others in every row, one of +inf above them.

    Returns (idx int32 [T, k], weights fp32 [T, k]), in descending order of the keys. The
    weights are differentiable with respect to the logits, once: a second derivative is
    refused when it is asked for, a forward-mode one at once.
    """
    if top_groups is None:
        top_groups = groups
    args = (logits, k, score, bias, groups, top_groups, group_top, renormalise, scale)
    if stream is not None or elsewhere(logits):
        return run_on(stream, route_experts, *args)
    refuse_tangents("route_experts", logits)
    if logits.requires_grad and torch.is_grad_enabled():
        return _RouteExperts.apply(*args)
    return _forward(*args)


def route_experts_backward(d_weights: torch.Tensor, logits: torch.Tensor, idx: torch.Tensor, score: str = "softmax",
                           renormalise: bool = True, scale: float = 1.0, stream: torch.cuda.Stream = None):
    """d_logits [T, E] in the logits' type from d_weights fp32 [T, k], with the idx that
    route_experts returned for these logits and the same score, renormalise and scale. It has
    no derivative itself, and refuses one when it is asked for."""
    if stream is not None or elsewhere(d_weights):
        return run_on(stream, route_experts_backward, d_weights, logits, idx, score, renormalise, scale)
    refuse_tangents("route_experts_backward", d_weights, logits)
    args = (d_weights, logits, idx, score, renormalise, scale)
    if torch.is_grad_enabled() and (d_weights.requires_grad or logits.requires_grad):
        return _RouteGradient.apply(*args)
    return _backward(*args)
