"""The example layer of routing, dispatch, 8-bit products and combine together, and the gradients of its trained form."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp8_layer.py")
    spec = importlib.util.spec_from_file_location("fp8_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_layer_against_the_plain_one():
    """A value v of [1, 2) in steps of 1/8 is off by 1/16 / sqrt(3) = 0.036 on an average, relative to it (the mean of
    1 / v^2 is 1/2) 2.55%, and so is a product of such rows with weights. The SwiGLU multiplies the errors of gate and up
    (silu is near g / 2 for the gates here, whose deviation is 0.45), and h is rounded once more: sqrt(3) 2.55% = 4.4% on an
    average over tokens. One token's five SwiGLUs have some 1,300 values, but the few largest blocks carry most of its
    norm: half as much again is allowed, 6.6%."""
    worst, norms = _example().main()
    assert worst < 0.066
    assert all(v > 0 for v in norms.values())


def test_the_layer_is_the_same_captured():
    ex = _example()
    import sparse_mixture_experts_gemv_gb300 as M
    layer = ex.make_layer()
    x = torch.randn(600, 512, generator=torch.Generator("cuda").manual_seed(3), device="cuda").bfloat16()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer.forward(x)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        held = layer.forward(x)
    for seed in (4, 5):
        x.copy_(torch.randn(600, 512, generator=torch.Generator("cuda").manual_seed(seed), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(held, layer.forward(x))
    assert M.fp8_sync_status() == M.MOE_OK


def test_gradients_against_differences():
    """The loss in 64 bits with the choices held: differences along a random direction of all parameters and the input."""
    ex = _example()
    import sparse_mixture_experts_gemv_gb300 as M
    model = ex.TrainedLayer(32, 6, 16, 2)
    g = torch.Generator("cuda").manual_seed(5)
    x = torch.randn(40, 32, generator=g, device="cuda", requires_grad=True)
    mix = torch.randn(40, 32, generator=g, device="cuda")
    (model(x) * mix).sum().backward()
    idx, _ = M.route_experts(x.detach() @ model.router.detach().T, 2)
    idx = idx.long()

    def loss(x, router, gate_up, down):
        top = (x @ router.T).softmax(1).gather(1, idx)
        w = top / top.sum(1, keepdim=True)
        out = torch.zeros_like(x)
        for j in range(2):
            a = torch.einsum("th,tfh->tf", x, gate_up[idx[:, j]])
            gate, up = a.chunk(2, dim=1)
            h = torch.nn.functional.silu(gate) * up
            out = out + w[:, j, None] * torch.einsum("ti,thi->th", h, down[idx[:, j]])
        return float((out * mix.double()).sum())

    leaves = [x, model.router, model.gate_up, model.down]
    at = [t.detach().double() for t in leaves]
    way = [torch.randn(t.shape, generator=g, device="cuda").double() for t in at]
    step = 1e-6
    want = (loss(*[a + step * d for a, d in zip(at, way)]) - loss(*[a - step * d for a, d in zip(at, way)])) / (2 * step)
    terms = torch.cat([(t.grad.double() * d).flatten() for t, d in zip(leaves, way)])
    # products of some tens of terms in 32 bits, a dozen roundings deep
    assert abs(float(terms.sum()) - want) < 1e-5 * float(terms.abs().sum())
