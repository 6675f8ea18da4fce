"""The down sums of int8_experts between the product and the weighted sum: held in 32 bits, whatever the
channels' scales are and however many tokens share the call."""
import numpy as np
import pytest

from oracle import route_int8_oracle as o
from test_gpu_int8 import _choices, _experts, _half, _np, _x

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _close(x, idx, w, ex, got):
    ref, mag, unsure = o.experts(_np(x), idx.cpu().numpy(), _np(w), *(_np(a) for a in ex))
    # 2^-17 of the magnitude of the terms: products' and scales' roundings (2^-24 each), SwiGLU (2^-20), sums over
    # I and k. Then the output's half step, and half a step of fp16 below its normal range.
    tol = 2.0 ** -17 * mag + unsure
    tol = tol + _half(x.dtype) * (np.abs(ref) + tol) + (2.0 ** -25 if x.dtype is torch.float16 else 1e-40)
    err = np.abs(_np(got) - ref)
    assert (err <= tol).all(), (float((err / tol).max()), np.argwhere(err > tol)[:4])
    return ref


@pytest.mark.parametrize("T", [3, 16, 17, 40, 200])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_the_output_rounds_once(T, dtype):
    import sparse_mixture_experts_gemv_gb300 as M
    x, (idx, w), ex = _x(T, 256, dtype, seed=T), _choices(T, 8, 4, seed=T), _experts(8, 256, 384)
    _close(x, idx, w, ex, M.int8_experts(x, idx, w, *ex))


@pytest.mark.parametrize("T", [3, 40, 200])
def test_channels_with_scales_far_below_their_experts_largest(T):
    """An output channel adds nothing but its own values up: its scale may be any part of its expert's largest."""
    import sparse_mixture_experts_gemv_gb300 as M
    x, (idx, w), ex = _x(T, 256, "bf16", seed=T), _choices(T, 8, 3, seed=T), _experts(8, 256, 384)
    for c, power in enumerate((0, -14, -24, -40, -90)):
        ex[3][:, c::5] *= 2.0 ** power
    ex[3][2] *= 2.0 ** 20            # an expert whose scales are far above the others'
    got = M.int8_experts(x, idx, w, *ex)
    ref = _close(x, idx, w, ex, got)
    assert (np.abs(ref[:, 4::5]).max(0) > 0).all()


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("scale", [float("inf"), float("nan"), 3e38, 1e-45])
def test_a_channel_of_any_scale_leaves_the_others_alone(T, scale):
    import sparse_mixture_experts_gemv_gb300 as M
    x, (idx, w), ex = _x(T, 128, "bf16", seed=T), _choices(T, 4, 2, seed=T), _experts(4, 128, 64)
    want = M.int8_experts(x, idx, w, *ex)
    ex[3][:, 77] = scale
    got = M.int8_experts(x, idx, w, *ex)
    others = [c for c in range(128) if c != 77]
    assert torch.equal(got[:, others], want[:, others])
    if scale == 1e-45:               # 2^-149, the least there is
        assert (got[:, 77].abs() < 1e-37).all()
    elif scale != 3e38:
        assert not torch.isfinite(got[:, 77]).any()


@pytest.mark.parametrize("T,k", [(6, 8), (7, 8), (2, 24), (16, 8), (16, 24)])
def test_few_tokens_that_share_experts(T, k):
    """On either side of the rule that goes by the bytes read again for choices of the same expert."""
    import sparse_mixture_experts_gemv_gb300 as M
    E = 8 if k == 8 else 24
    x, (idx, w), ex = _x(T, 2048, "bf16", seed=T), _choices(T, E, k, seed=T), _experts(E, 2048, 512)
    idx[T - 1, 0] = -1
    _close(x, idx, w, ex, M.int8_experts(x, idx, w, *ex))
