"""The oracle of the token and 8-bit floating-point operators by brute force, and what the C entry points and the
Python calls refuse before anything reaches a device."""
import contextlib
import types

import numpy as np
import pytest

from oracle import tokens_fp8_oracle as o

torch = pytest.importorskip("torch")


def test_e4m3_codes_are_torchs():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(o.E4M3, want)


def test_rounding_to_e4m3_is_the_nearest_value_by_search():
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.normal(size=500) * 10.0 ** rng.integers(-4, 3, 500), (o._POSITIVE[1:] + o._POSITIVE[:-1]) / 2,
                        [0.0, -0.0, 448.0, 1e9, -1e9, 2.0 ** -10, 3 * 2.0 ** -10, np.nan]])
    codes = o.to_e4m3(v)
    for x, c in zip(v, codes):
        if np.isnan(x):
            assert c == 127
            continue
        far = np.abs(o._POSITIVE - min(abs(x), 448.0))
        best = [i for i in range(127) if far[i] == far.min()]
        assert c & 127 == (best[0] if len(best) == 1 else next(i for i in best if i % 2 == 0))
        assert (c >> 7) == np.signbit(x)


def test_quantization_and_product_by_hand():
    x = np.zeros((1, 256))
    x[0, 0], x[0, 1], x[0, 200] = 448.0, 3.3, -2.0
    codes, scales = o.quantize(x)
    one = float(np.float32(448) * np.float32(1 / 448))   # the rounded reciprocal's product, next to 1
    assert abs(scales[0, 0] - 1) < 1e-6 and scales[0, 0] == np.float32(one)
    assert o.E4M3[codes[0, 0]] == 448 and o.E4M3[codes[0, 1]] == 3.25 and o.E4M3[codes[0, 200]] == -448
    w = np.ones((130, 256))
    w_scale = np.array([[1.0, 2.0], [3.0, 4.0]])
    out, mag = o.matmul(o.E4M3[codes], scales, w, w_scale)
    a, b = (448 + 3.25) * float(scales[0, 0]), -448.0 * float(scales[0, 1])
    np.testing.assert_allclose(out[0, [0, 129]], [a + 2 * b, 3 * a + 4 * b], rtol=1e-12)
    np.testing.assert_allclose(mag[0, 0], a - 2 * b, rtol=1e-12)


def test_places_and_sums_by_hand():
    idx = np.array([[2, 0], [0, -1], [2, 2]])
    offsets, pos = o.places(idx, 3)
    assert offsets.tolist() == [0, 2, 2, 5]
    assert pos.tolist() == [[2, 0], [1, ~5], [3, 4]]
    x = np.array([[1.0], [2.0], [3.0]])
    assert o.dispatch(x, pos)[:, 0].tolist() == [1, 2, 1, 3, 3, 0]
    y = np.arange(6.0)[:, None] + 1
    w = np.array([[0.5, 2.0], [1.0, 7.0], [1.0, 1.0]])
    assert o.combine(y, pos, w)[0][:, 0].tolist() == [3 * 0.5 + 2.0, 2.0, 4.0 + 5.0]
    d_y, d_w, _ = o.combine_backward(x, y, pos, w)
    assert d_y[:, 0].tolist() == [2.0, 2.0, 0.5, 3.0, 3.0, 0.0]
    assert d_w.tolist() == [[3.0, 1.0], [4.0, 0.0], [12.0, 15.0]]


FAKE = 0x10000   # never read: every call below is refused first


def test_the_c_calls_refuse_bad_arguments_before_touching_the_device():
    import ctypes
    from sparse_mixture_experts_gemv_gb300 import _native as N
    L, bad, out = N.load(), N.MOE_ERR_INVALID_ARG, N.MOE_ERR_UNSUPPORTED
    far = [FAKE + (i << 32) for i in range(8)]

    def dispatch(x=far[0], row=64, stride=64, xs=None, scales=0, idx=far[1], T=4, k=2, E=8, rows=far[2], rs=None,
                 offsets=far[3], pos=far[4], ws=None, nb=0):
        return L.moe_dispatch_tokens(x, row, stride, xs, scales, idx, T, k, E, rows, rs, offsets, pos, ws, nb, None)
    assert [dispatch(T=-1), dispatch(k=0), dispatch(E=0), dispatch(row=0), dispatch(stride=63), dispatch(x=None),
            dispatch(idx=None), dispatch(rows=None), dispatch(offsets=None), dispatch(pos=None), dispatch(idx=far[1] + 2),
            dispatch(xs=far[5]), dispatch(scales=3), dispatch(xs=far[5], scales=3), dispatch(rows=far[0] + 16),
            dispatch(pos=far[1] + 4), dispatch(T=20000), dispatch(T=20000, ws=far[6], nb=100),
            dispatch(T=20000, ws=far[6] + 16, nb=1 << 20)] == [bad] * 19
    assert [dispatch(k=33), dispatch(E=1025), dispatch(T=1 << 29, k=4)] == [out] * 3

    def combine(y=far[0], dtype=1, stride=64, pos=far[1], w=far[2], T=4, k=2, H=64, out_=far[3]):
        return L.moe_combine_tokens(y, dtype, stride, pos, w, T, k, H, out_, None)
    assert [combine(y=None), combine(pos=None), combine(out_=None), combine(dtype=3), combine(dtype=4), combine(stride=63),
            combine(k=0), combine(H=0), combine(T=-1), combine(y=far[0] + 1), combine(w=far[2] + 2),
            combine(out_=far[0] + 64)] == [bad] * 12
    assert combine(k=33) == out and combine(T=0, y=None) == N.MOE_OK

    def back(d=far[0], ds=64, y=far[1], dtype=1, ys=64, pos=far[2], w=far[3], T=4, k=2, H=64, dy=far[4], dw=far[5]):
        return L.moe_combine_tokens_backward(d, ds, y, dtype, ys, pos, w, T, k, H, dy, dw, None)
    assert [back(d=None), back(y=None), back(pos=None), back(ds=63), back(ys=63), back(dtype=5), back(k=0),
            back(dy=far[0] + 32), back(dy=far[1] + 32), back(dw=far[5] + 1)] == [bad] * 10
    assert back(k=33) == out and back(T=0) == N.MOE_OK and back(dy=None, dw=None) == N.MOE_OK

    def quantize(x=far[0], dtype=1, stride=64, swiglu=0, T=4, K=64, q=far[1], s=far[2]):
        return L.moe_block_quantize(x, dtype, stride, swiglu, T, K, q, s, None)
    assert [quantize(x=None), quantize(q=None), quantize(s=None), quantize(dtype=3), quantize(dtype=4), quantize(stride=56),
            quantize(swiglu=1), quantize(stride=65), quantize(x=far[0] + 2), quantize(q=far[1] + 8), quantize(T=-1),
            quantize(K=0), quantize(q=far[0] + 64)] == [bad] * 13
    assert [quantize(K=24, stride=24), quantize(K=65552, stride=65552)] == [out] * 2 and quantize(T=0, x=None) == N.MOE_OK

    def matmul(x=far[0], dtype=4, xst=64, xs=far[1], w=far[2], wst=64, ws=far[3], y=far[4], od=1, T=4, n=8, K=64, sc=None,
               nb=0):
        return L.moe_block_matmul(x, dtype, xst, xs, w, wst, ws, y, od, T, n, K, sc, nb, None)
    assert [matmul(x=None), matmul(w=None), matmul(ws=None), matmul(y=None), matmul(xs=None), matmul(dtype=1),
            matmul(dtype=3), matmul(od=4), matmul(xst=48), matmul(wst=48), matmul(xst=72), matmul(x=far[0] + 8),
            matmul(y=far[4] + 1), matmul(y=far[0]), matmul(y=far[2]), matmul(T=20, dtype=1, xs=None),
            matmul(T=20, dtype=1, xs=None, sc=far[5], nb=511),
            matmul(T=20, dtype=1, xs=None, sc=far[5] + 16, nb=4096)] == [bad] * 18
    assert matmul(K=40) == out and matmul(T=0, x=None) == N.MOE_OK and matmul(n=0, x=None) == N.MOE_OK

    def grouped(off=far[5], E=4, M=4, n=8, K=64, y=far[4]):
        return L.moe_block_grouped_matmul(far[0], 4, K, far[1], off, far[2], far[3], y, 1, M, E, n, K, None, 0, None)
    assert [grouped(off=None), grouped(off=far[5] + 2), grouped(E=0), grouped(M=-1), grouped(y=far[2] + 1000)] == [bad] * 5
    assert [grouped(E=1025), grouped(K=40)] == [out] * 2 and grouped(M=0) == N.MOE_OK

    b = ctypes.c_int64(7)
    assert L.moe_block_matmul_workspace(3, 144, 4, ctypes.byref(b)) == N.MOE_OK and b.value == 0
    assert L.moe_block_matmul_workspace(17, 144, 1, ctypes.byref(b)) == N.MOE_OK and b.value == 2560 + 256
    assert L.moe_block_matmul_workspace(5, 4096, 1, ctypes.byref(b)) == N.MOE_OK and b.value == 0
    assert L.moe_block_matmul_workspace(16, 1296, 1, ctypes.byref(b)) == N.MOE_OK and b.value == 20736 + 768
    assert L.moe_block_matmul_workspace(1, 4112, 1, ctypes.byref(b)) == N.MOE_OK and b.value == 4352 + 256
    assert L.moe_block_matmul_workspace(3, 144, 3, ctypes.byref(b)) == bad
    assert L.moe_block_matmul_workspace(3, 144, 1, None) == bad


def test_the_python_calls_scratch_is_the_librarys():
    import ctypes
    from sparse_mixture_experts_gemv_gb300 import _native as N, fp8
    b = ctypes.c_int64()
    for rows, K in ((1, 16), (3, 144), (5, 4096), (6, 4096), (16, 1280), (17, 64), (1, 4112), (333, 2560), (65536, 4096), (7, 65536)):
        for code in (0, 1, 2):
            assert N.load().moe_block_matmul_workspace(rows, K, code, ctypes.byref(b)) == N.MOE_OK
            inside = rows <= 16 and K <= 4096 and rows * K <= 20480
            assert b.value == (0 if inside else fp8._pad256(rows * K) + fp8._pad256(rows * fp8._blocks(K) * 4))


class Stand:
    """A CUDA tensor as far as the calls look before they run anything."""

    is_cuda, requires_grad = True, False

    def __init__(self, index):
        self.device = torch.device("cuda", index)

    def get_device(self):
        return self.device.index


class Entered(Exception):
    pass


CALLS = {"dispatch_tokens": lambda M, t, **kw: M.dispatch_tokens(t, t, 4, **kw),
         "dispatch_tokens_backward": lambda M, t, **kw: M.dispatch_tokens_backward(t, t, **kw),
         "combine_tokens": lambda M, t, **kw: M.combine_tokens(t, t, t, **kw),
         "combine_tokens_backward": lambda M, t, **kw: M.combine_tokens_backward(t, t, t, t, **kw),
         "fp8_quantize": lambda M, t, **kw: M.fp8_quantize(t, **kw),
         "fp8_matmul": lambda M, t, **kw: M.fp8_matmul(t, t, t, **kw),
         "fp8_grouped_matmul": lambda M, t, **kw: M.fp8_grouped_matmul(t, t, t, t, **kw)}


def _switch_to(where):
    def guard(device):
        raise Entered(where, device)
    return guard


@pytest.mark.parametrize("call", list(CALLS))
def test_the_tensors_device_becomes_the_current_one(call, monkeypatch):
    import sparse_mixture_experts_gemv_gb300 as M
    from sparse_mixture_experts_gemv_gb300 import _tensors
    monkeypatch.setattr(_tensors, "_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", _switch_to("device"))
    with pytest.raises(Entered) as e:
        CALLS[call](M, Stand(1))
    assert e.value.args == ("device", torch.device("cuda", 1))
    with pytest.raises(AttributeError):      # on the current one it goes on at once, to what a stand-in has not
        CALLS[call](M, Stand(0))


@pytest.mark.parametrize("call", list(CALLS))
def test_a_stream_of_another_device_is_refused(call, monkeypatch):
    import sparse_mixture_experts_gemv_gb300 as M
    from sparse_mixture_experts_gemv_gb300 import _tensors
    monkeypatch.setattr(_tensors, "_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", _switch_to("stream"))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: None)
    stream = types.SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream"):
        CALLS[call](M, Stand(0), stream=stream)
    with pytest.raises(Entered) as e:
        CALLS[call](M, Stand(1), stream=stream)
    assert e.value.args == ("stream", stream)


def test_the_status_is_read_on_the_streams_device(monkeypatch):
    import sparse_mixture_experts_gemv_gb300 as M
    from sparse_mixture_experts_gemv_gb300 import fp8
    current, seen = [0], []

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], d.index
        yield
        current[0] = before

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(fp8.N, "load", lambda: types.SimpleNamespace(
        moe_block_sync_status=lambda s: seen.append((s, current[0])) or 0))
    assert M.fp8_sync_status(types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=77)) == 0
    assert seen == [(77, 1)] and current == [0]


def test_inputs_that_would_lose_a_gradient_or_a_tangent_are_refused():
    import sparse_mixture_experts_gemv_gb300 as M
    from torch.autograd import forward_ad
    x, leaf, idx = torch.ones(2, 16), torch.ones(2, 16, requires_grad=True), torch.zeros(2, 1, dtype=torch.int32)
    for call in (lambda: M.fp8_quantize(leaf), lambda: M.fp8_matmul(leaf, x, x), lambda: M.fp8_matmul(x, x, leaf),
                 lambda: M.fp8_matmul(x, x, x, leaf), lambda: M.fp8_grouped_matmul(leaf, idx, x, x),
                 lambda: M.fp8_grouped_matmul(x, idx, x, leaf), lambda: M.dispatch_tokens(leaf, idx, 4, x),
                 lambda: M.dispatch_tokens(x, idx, 4, leaf),
                 lambda: M.dispatch_tokens(x.to(torch.float8_e4m3fn).requires_grad_(), idx, 4)):
        with pytest.raises(ValueError, match="gradient"):
            call()
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, x)
        for call in (lambda: M.dispatch_tokens(dual, idx, 4), lambda: M.combine_tokens(dual, idx, x),
                     lambda: M.combine_tokens(x, idx, dual), lambda: M.dispatch_tokens_backward(dual, idx),
                     lambda: M.combine_tokens_backward(dual, x, idx, x), lambda: M.fp8_quantize(dual)):
            with pytest.raises(ValueError, match="tangent"):
                call()


def test_tensors_of_the_host_are_refused():
    import sparse_mixture_experts_gemv_gb300 as M
    x, idx = torch.ones(2, 16), torch.zeros(2, 1, dtype=torch.int32)
    for call in (lambda: M.dispatch_tokens(x, idx, 4), lambda: M.dispatch_tokens_backward(x, idx),
                 lambda: M.combine_tokens(x, idx, x), lambda: M.combine_tokens(x, idx, None),
                 lambda: M.combine_tokens_backward(x, x, idx, x), lambda: M.fp8_quantize(x),
                 lambda: M.fp8_matmul(x, x, x), lambda: M.fp8_grouped_matmul(x, idx, x, x),
                 lambda: M.fp8_grouped_matmul(x, None, x, x)):
        with pytest.raises(ValueError):
            call()


def test_weights_that_would_lose_a_gradient_or_a_tangent_are_refused():
    """A parameter of float8_e4m3fn requires a gradient unless it is told not to."""
    import sparse_mixture_experts_gemv_gb300 as M
    from torch.autograd import forward_ad
    x, idx = torch.ones(2, 16), torch.zeros(2, 1, dtype=torch.int32)
    w = torch.nn.Parameter(torch.ones(2, 16).to(torch.float8_e4m3fn))
    assert w.requires_grad
    calls = (lambda w: M.fp8_matmul(x, w, x), lambda w: M.fp8_matmul(x, w, x, x), lambda w: M.fp8_grouped_matmul(x, idx, w, x))
    for call in calls:
        with pytest.raises(ValueError, match="gradient"):
            call(w)
        with torch.no_grad(), pytest.raises(ValueError, match="must be"):   # goes on to the other checks
            call(w)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(w.detach(), w.detach())
        for call in calls:
            with pytest.raises(ValueError, match="tangent"):
                call(dual)
