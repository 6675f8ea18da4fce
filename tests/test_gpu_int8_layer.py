"""The example layer: routing, int8 experts and an int8 shared expert together."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "int8_layer.py")
    spec = importlib.util.spec_from_file_location("int8_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_layer_against_the_plain_one():
    """A value rounded to 1/127 of its row's largest is off by at most half of that; a row of 512 normals
    reaches about 3.5 deviations, so activations are off by 3.5 / 127 / sqrt(12) = 0.8% twice over on the way."""
    worst, before, after = _example().main()
    assert worst < 0.02
    assert after < before


def test_gradient_of_the_router_against_differences():
    ex = _example()
    layer, _ = ex.make_layer(H=256, E=32, I=64)
    x = torch.randn(40, 256, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    d = torch.randn(40, 4, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    _, (idx, _) = layer.route(x)
    grad = layer.router_gradient(x, d).double()
    direction = torch.randn(256, 32, device="cuda", generator=torch.Generator("cuda").manual_seed(4)).double()

    def loss(step):
        s = torch.sigmoid(x.double() @ (layer.router.double() + step * direction)).gather(1, idx.long())
        return float((2.5 * s / s.sum(1, keepdim=True) * d.double()).sum())

    step = 1e-6
    want = (loss(step) - loss(-step)) / (2 * step)
    got = float((grad * direction).sum())
    # logits in 32 bits with sums over 256, and the gradient's own roundings
    assert abs(got - want) < 1e-4 * float((grad * direction).abs().sum())
