"""route_experts under a bias that is not finite, or as large as fp32 goes: NaN counts as -inf, +inf as the
largest finite value, and an expert whose key is -inf ranks below all others. Every output is written."""
import numpy as np
import pytest

from test_gpu_route_experts import _check, _make

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

INF, NAN = float("inf"), float("nan")
MAX = torch.finfo(torch.float32).max


def _biases(E):
    base = torch.linspace(-0.1, 0.1, E)
    out = {"one forced": {E // 2: INF}, "several forced": {0: INF, E // 3: INF, E - 1: INF}, "one off": {1: -INF},
           "one NaN": {E - 2: NAN}, "mixed": {0: NAN, 1: INF, 2: -INF, E - 1: MAX}, "lowest": {0: -MAX, E // 2: -MAX}}
    made = {"all forced": torch.full((E,), INF), "all NaN": torch.full((E,), NAN), "all off": torch.full((E,), -INF),
            "all lowest": torch.full((E,), -MAX), "all largest": torch.full((E,), MAX)}
    for name, at in out.items():
        made[name] = base.clone()
        for e, v in at.items():
            made[name][e] = v
    half = base.clone()
    half[: E // 2] = -INF
    half[E // 2:E // 2 + E // 4] = -MAX
    made["halves"] = half
    run = base.clone()
    run[:max(2, E // 4)] = NAN       # whole lanes of a warp
    made["a run of NaN"] = run
    return made


@pytest.mark.parametrize("E", [8, 60, 128, 256, 512])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_biases_that_are_not_finite(E, score):
    logits = _make(9, E, "fp32", E)
    logits[3, 1::3] = -INF
    logits[4] = -INF
    logits[5, 2] = NAN
    for name, bias in _biases(E).items():
        for k in (1, 2, 4):
            for groups, top, group_top in ((1, 1, 2), (4, 2, 2), (4, 2, 1), (4, 3, 2)):
                # what the allocator hands out next holds numbers that are no choice
                torch.full((9, k), -77, dtype=torch.int32, device="cuda")
                _check(logits, k, score=score, bias=bias.cuda(), groups=groups, top_groups=top, group_top=group_top,
                       renormalise=k > 1)


def test_groups_all_masked_rank_above_groups_that_are_off():
    """Two keys of the lowest value add up to more than none."""
    x = torch.zeros(2, 16, device="cuda")
    x[0, :4] = -INF
    bias = torch.full((16,), -MAX, device="cuda")
    for score in ("softmax", "sigmoid"):
        idx, _ = _check(x, 4, score=score, bias=bias, groups=4, top_groups=1)
        assert idx[0].tolist() == [4, 5, 6, 7] and idx[1].tolist() == [0, 1, 2, 3]


def test_sums_of_two_largest_keys():
    """A group of two forced experts before a group with one, whichever comes first."""
    x = torch.randn(4, 32, generator=torch.Generator().manual_seed(1)).cuda()
    bias = torch.zeros(32, device="cuda")
    bias[3] = INF
    bias[20] = bias[21] = INF
    for score in ("softmax", "sigmoid"):
        idx, _ = _check(x, 2, score=score, bias=bias, groups=4, top_groups=1)
        assert (idx == torch.tensor([20, 21], device="cuda")).all()
