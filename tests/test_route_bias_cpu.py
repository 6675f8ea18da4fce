"""The oracle's choice under biases that are not finite, on worked examples."""
import pytest

from oracle import route_int8_oracle as o

INF, NAN = float("inf"), float("nan")
MAX = 3.4028234663852886e38


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_that_are_not_finite(score):
    x = [1.0, 3.0, 2.0, 0.0]
    assert o.choose(x, 2, score, bias=[0, 0, 0, INF]) == [3, 1]
    assert o.choose(x, 4, score, bias=[INF, 0, 0, MAX]) == [0, 3, 1, 2]       # both count the same: by index
    assert o.choose(x, 4, score, bias=[0, NAN, 0, 0]) == [2, 0, 3, 1]
    assert o.choose(x, 4, score, bias=[-INF, NAN, 0, -MAX]) == [2, 3, 0, 1]
    assert o.choose([1.0, -INF, 2.0, 0.0], 4, score, bias=[NAN] * 4) == [0, 1, 2, 3]
    # a group of two of the lowest value before one that is off, and two forced before one
    assert o.choose([-INF, -INF, 1.0, 2.0], 2, score, bias=[0, 0, -MAX, -MAX], groups=2, top_groups=1) == [2, 3]
    assert o.choose(x, 2, score, bias=[INF, 0, INF, INF], groups=2, top_groups=1) == [2, 3]
