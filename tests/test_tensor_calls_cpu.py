"""What the calls on torch tensors do before anything reaches a device, with stand-ins for the tensors and the
current device: the tensors' own device becomes the current one, a stream of another device is refused."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")


class Stand:
    """A CUDA tensor as far as the calls look before they run anything."""

    is_cuda, requires_grad = True, False

    def __init__(self, index):
        self.device = torch.device("cuda", index)

    def get_device(self):
        return self.device.index


class Entered(Exception):
    pass


CALLS = {"route_experts": lambda M, t, **kw: M.route_experts(t, 2, **kw),
         "route_experts_backward": lambda M, t, **kw: M.route_experts_backward(t, t, t, **kw),
         "int8_matmul": lambda M, t, **kw: M.int8_matmul(t, t, t, **kw),
         "int8_experts": lambda M, t, **kw: M.int8_experts(t, t, t, t, t, t, t, **kw)}


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
    from sparse_mixture_experts_gemv_gb300 import int8
    current, seen = [0], []

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], d.index
        yield
        current[0] = before

    monkeypatch.setattr(torch.cuda, "device", device)
    lib = types.SimpleNamespace(moe_quant_sync_status=lambda s: seen.append((s, current[0])) or 0)
    monkeypatch.setattr(int8.N, "load", lambda: lib)
    assert M.int8_sync_status(types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=77)) == 0
    assert seen == [(77, 1)] and current == [0]


def test_tangents_are_refused():
    from torch.autograd import forward_ad
    from sparse_mixture_experts_gemv_gb300 import _tensors
    x = torch.ones(3)
    _tensors.refuse_tangents("call", x, None)
    with forward_ad.dual_level():
        _tensors.refuse_tangents("call", x, None)
        with pytest.raises(ValueError, match="tangent"):
            _tensors.refuse_tangents("call", x, None, forward_ad.make_dual(x, x))


def test_inputs_that_record_a_gradient_are_refused():
    from sparse_mixture_experts_gemv_gb300 import _tensors
    x, leaf = torch.ones(3), torch.ones(3, requires_grad=True)
    _tensors.refuse_gradients("call", x, None)
    for t in (leaf, leaf * 2):
        with pytest.raises(ValueError, match="gradient"):
            _tensors.refuse_gradients("call", x, None, t)
        with torch.no_grad():
            _tensors.refuse_gradients("call", x, None, t)
    _tensors.refuse_gradients("call", leaf.detach())


def test_the_products_refuse_before_they_look_at_types():
    import sparse_mixture_experts_gemv_gb300 as M
    x, leaf = torch.ones(2, 16), torch.ones(2, 16, requires_grad=True)
    for args in ((leaf, x, x), (x, x, leaf), (x, x, x, leaf)):
        with pytest.raises(ValueError, match="gradient"):
            M.int8_matmul(*args)
    for at in (0, 2, 4, 6):
        with pytest.raises(ValueError, match="gradient"):
            M.int8_experts(*[leaf if i == at else x for i in range(7)])


def test_the_allocator_learns_of_both_streams(monkeypatch):
    from sparse_mixture_experts_gemv_gb300 import _tensors
    device = torch.device("cuda", 0)
    theirs, ours = types.SimpleNamespace(device=device, at=1), types.SimpleNamespace(device=device, at=2)
    seen = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: ours)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch, "Tensor", Stand)
    monkeypatch.setattr(Stand, "record_stream", lambda t, s: seen.append((t, s)), raising=False)
    a, b, c, d = (Stand(0) for _ in range(4))
    assert _tensors.run_on(theirs, lambda *args: c, a, 3, b, None) is c
    assert seen == [(a, theirs), (b, theirs), (c, ours)]
    seen.clear()
    assert _tensors.run_on(theirs, lambda *args: (c, d), a) == (c, d)
    assert seen == [(a, theirs), (c, ours), (d, ours)]
    seen.clear()
    _tensors.run_on(ours, lambda *args: c, a)
    assert seen == []


@pytest.mark.parametrize("K", [1024, 49168, 65536])
def test_more_rows_than_a_grids_second_dimension(K):
    """The dot-product kernel takes a row or more a CTA there: what may not fit needs the other one's workspace."""
    import ctypes
    from sparse_mixture_experts_gemv_gb300 import _native as N
    need = ctypes.c_int64()
    ws = N.load().moe_quant_matmul_workspace
    assert ws(65536, 1, K, N.MOE_DTYPE_S8, ctypes.byref(need)) == N.MOE_OK and need.value > 65536 * K
    assert ws(65535, 1, K, N.MOE_DTYPE_S8, ctypes.byref(need)) == N.MOE_OK and need.value == 0


def test_a_routing_rule_is_kept_by_its_values():
    """A tensor among them would be found again by its identity, with what it held the first time."""
    from sparse_mixture_experts_gemv_gb300.routing import _config
    plain = (64, 4, "softmax", 1, 1, 2, True, 2.0)
    assert _config(*plain)._obj.scale == 2.0 and _config(*plain[:7], 3)._obj.scale == 3.0
    scale = torch.tensor(2.0)
    for at, t in ((7, scale), (7, scale.clone().requires_grad_()), (6, torch.tensor(True)), (1, torch.tensor(4))):
        for _ in range(2):
            with pytest.raises(ValueError, match="tensor"):
                _config(*[t if i == at else v for i, v in enumerate(plain)])
    for at, n in ((1, -1), (1, 2 ** 32 + 4), (3, 2 ** 32 + 1), (4, 2 ** 31), (5, 2 ** 40 + 2)):
        with pytest.raises(ValueError, match="31 bits"):
            _config(*[n if i == at else v for i, v in enumerate(plain)])
