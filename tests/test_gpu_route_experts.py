"""route_experts and its gradient against the fp64 oracle: choices equal, weights and
gradients within the rounding of 32 bits."""
import numpy as np
import pytest

from oracle import route_int8_oracle as o

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

INF = float("inf")
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}

# exp to 2 units in the last place, its argument's rounding (spreads up to 64: 2^-18), sums of at
# most 512 terms in a tree of 16 + 5, quotients: 2^-16 covers them all
REL = 2.0 ** -16


def _make(T, E, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * spread).to(DT[dtype]).cuda()


def _check(logits, k, **kw):
    import sparse_mixture_experts_gemv_gb300 as M
    bias = kw.pop("bias", None)
    idx, w = M.route_experts(logits, k, bias=bias, **kw)
    assert idx.dtype is torch.int32 and w.dtype is torch.float32 and idx.shape == w.shape == (len(logits), k)
    x = logits.float().cpu().numpy()
    b = None if bias is None else bias.cpu().numpy()
    kw.setdefault("top_groups", kw.get("groups", 1))
    ri, rw = o.route(x, k, bias=b, **kw)
    got = idx.cpu().numpy()
    bad = np.argwhere((got != ri).any(1))[:, 0] if k else []
    assert len(bad) == 0, (bad[:5], got[bad[:3]], ri[bad[:3]])
    err = np.abs(w.cpu().numpy() - rw)
    assert (err <= REL * np.abs(rw) + 1e-37).all(), (err / np.maximum(rw, 1e-30)).max()
    return idx, w


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (5, 3), (16, 2), (33, 8), (60, 4), (64, 6), (100, 7), (128, 8),
                                 (160, 6), (256, 8), (257, 9), (384, 8), (500, 32), (512, 8)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_top_k_of_the_scores(E, k, dtype):
    for score in ("softmax", "sigmoid"):
        for renormalise in (True, False):
            _check(_make(37, E, dtype, E + k), k, score=score, renormalise=renormalise, scale=1.5)


@pytest.mark.parametrize("E,groups,top,k", [(8, 2, 1, 4), (12, 4, 2, 6), (60, 4, 3, 5), (64, 32, 4, 8), (160, 8, 3, 6),
                                            (256, 8, 4, 8), (256, 8, 8, 8), (384, 3, 2, 8), (512, 8, 4, 8),
                                            (512, 16, 1, 32), (500, 25, 5, 10), (32, 32, 7, 7)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_and_bias(E, groups, top, k, score):
    for dtype in ("fp32", "bf16"):
        logits = _make(29, E, dtype, E * groups)
        bias = (torch.randn(E, generator=torch.Generator().manual_seed(7)) * 0.1).cuda()
        for b in (None, bias, (bias * 100).round() / 1000):
            for group_top in (1, 2):
                _check(logits, k, score=score, bias=b, groups=groups, top_groups=top, group_top=group_top)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 127, 1025, 20011])
def test_row_counts(T):
    _check(_make(T, 64, "fp32", T), 4, score="sigmoid", bias=torch.linspace(-0.1, 0.1, 64).cuda(), groups=4, top_groups=2)


def test_no_rows():
    import sparse_mixture_experts_gemv_gb300 as M
    idx, w = M.route_experts(torch.empty(0, 16, device="cuda"), 2)
    assert idx.shape == w.shape == (0, 2)
    assert M.route_experts_backward(w, torch.empty(0, 16, device="cuda"), idx).shape == (0, 16)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("keyed", [False, True])
def test_experts_that_are_off_and_infinities(score, keyed):
    x = _make(12, 48, "fp32", 5)
    x[0] = -INF                                   # nothing on
    x[1, 3:] = -INF                               # fewer on than chosen
    x[2, ::2] = float("nan")
    x[3] = float("nan")
    x[4, 7] = INF                                 # counts as the largest finite value
    x[5, 7:9] = INF
    x[6] = torch.finfo(torch.float32).min         # the lowest value is a value
    x[6, 5] = -INF
    x[7, :24] = torch.finfo(torch.float32).min
    x[8] = 0.0
    x[8, ::3] = -0.0                              # equal to 0
    x[9, 30] = -INF
    x[10, 16:] = -INF                             # whole groups off
    bias = torch.full((48,), 0.25, device="cuda") if keyed else None
    if keyed:
        bias[30] = 9.0                            # an expert that is off stays off
    for renormalise in (True, False):
        idx, w = _check(x, 5, score=score, bias=bias, renormalise=renormalise, scale=2.0)
        assert (w[0] == 0).all() and (w[3] == 0).all() and torch.isfinite(w).all()
        _check(x, 5, score=score, bias=bias, renormalise=renormalise, groups=3, top_groups=2, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_keys_closer_than_32_bits(score):
    """Every expert's key within a few 1e-9 of the others: the order is decided in 64 bits."""
    rng = np.random.default_rng(11)
    E = 96
    x = rng.normal(size=(64, E)).astype(np.float32)
    for t in range(len(x)):
        s, _ = o.scores(x[t], score)
        x[t, :] = x[t]
        bias = (0.9 - s).astype(np.float32) if t == 0 else bias
    x[1:] = x[0] + rng.normal(size=(63, E)).astype(np.float32) * 1e-7
    logits, b = torch.from_numpy(x).cuda(), torch.from_numpy(bias).cuda()
    for kw in ({}, {"groups": 4, "top_groups": 2}, {"groups": 4, "top_groups": 2, "group_top": 1}):
        import sparse_mixture_experts_gemv_gb300 as M
        idx, _ = M.route_experts(logits, 8, score=score, bias=b, **kw)
        got = idx.cpu().numpy()
        for t in range(len(x)):
            ri = o.choose(x[t], 8, score, bias, kw.get("groups", 1), kw.get("top_groups", 1), kw.get("group_top", 2))
            if list(got[t]) != ri:   # keys within 64 bits' rounding of each other may go either way
                s, _ = o.scores(x[t], score)
                key = s + bias.astype(np.float64)
                assert np.allclose(np.sort(key[got[t]]), np.sort(key[ri]), rtol=0, atol=1e-15), t


def test_equal_logits_go_by_index():
    x = torch.zeros(3, 512, device="cuda")
    idx, w = _check(x, 8, score="softmax")
    assert idx[0].tolist() == list(range(8))
    idx, _ = _check(x, 8, score="sigmoid", bias=torch.zeros(512, device="cuda"), groups=8, top_groups=3)
    assert idx[2].tolist() == list(range(8))
    _check((_make(501, 512, "fp32", 3) * 2).round(), 8, score="sigmoid", groups=8, top_groups=4,
           bias=torch.zeros(512, device="cuda"))


@pytest.mark.parametrize("spread", [30.0, 200.0])
def test_wide_logits(spread):
    x = _make(41, 128, "fp32", 9, spread)
    for score in ("softmax", "sigmoid"):
        import sparse_mixture_experts_gemv_gb300 as M
        idx, w = M.route_experts(x, 6, score=score)
        ri, rw = o.route(x.cpu().numpy(), 6, score)
        assert (idx.cpu().numpy() == ri).all()
        # arguments of exp up to 2^10: their rounding alone is 2^-14 of the result
        assert np.allclose(w.cpu().numpy(), rw, rtol=2.0 ** -13, atol=1e-37)


def test_rows_apart_and_off_16_byte_boundaries():
    base = _make(50, 131, "fp32", 21)
    for view in (base[:, :128], base[:, 1:129], base[:, 3:67], base.bfloat16()[:, 1:65], base[::2, 2:66],
                 base[:, :128].t().contiguous().t(), base[:1, 1:65]):
        _check(view, 6, score="sigmoid", bias=torch.linspace(0, 0.2, view.shape[1]).cuda())


def test_another_stream_and_repeats():
    import sparse_mixture_experts_gemv_gb300 as M
    x = _make(3000, 256, "bf16", 2)
    want = M.route_experts(x, 8, score="sigmoid")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        got = M.route_experts(x, 8, score="sigmoid", stream=s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


# ------------------------------------------------------------------------------------------ gradient
def _check_grad(logits, k, score, renormalise, scale, seed=0, **kw):
    import sparse_mixture_experts_gemv_gb300 as M
    idx, w = M.route_experts(logits, k, score=score, renormalise=renormalise, scale=scale, **kw)
    d = torch.randn(w.shape, generator=torch.Generator().manual_seed(seed)).cuda()
    got = M.route_experts_backward(d, logits, idx, score, renormalise, scale)
    assert got.dtype is logits.dtype and got.shape == logits.shape
    ref, mag = o.route_backward(d.cpu().numpy(), logits.float().cpu().numpy(), idx.cpu().numpy(), score, renormalise,
                                scale)
    half = 0.0 if logits.dtype is torch.float32 else torch.finfo(logits.dtype).eps / 2
    small = 2.0 ** -25 if logits.dtype is torch.float16 else 1e-37
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= REL * mag + half * np.abs(ref) + small).all(), (err / np.maximum(mag, 1e-30)).max()
    return idx, d, got


@pytest.mark.parametrize("E,k", [(1, 1), (5, 2), (16, 3), (60, 4), (129, 8), (256, 8), (512, 32)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_gradient(E, k, dtype, score, renormalise):
    _check_grad(_make(43, E, dtype, E), k, score, renormalise, 2.5)


def test_gradient_of_odd_rows_views_and_masks():
    base = _make(50, 131, "fp32", 31)
    base[3, ::2] = -INF
    base[4] = -INF
    base[5, 9] = float("nan")
    base[6, 11] = INF
    for view in (base[:, :128], base[:, 1:129], base[::3, 2:66], base.half()[:, 1:65]):
        for score in ("softmax", "sigmoid"):
            for renormalise in (True, False):
                _, _, got = _check_grad(view, 6, score, renormalise, 1.0)
                assert torch.isfinite(got).all()


def test_choices_outside_have_no_gradient():
    import sparse_mixture_experts_gemv_gb300 as M
    x = _make(2, 16, "fp32", 1)
    idx = torch.tensor([[3, -1], [16, 2 ** 30]], dtype=torch.int32, device="cuda")
    d = torch.ones(2, 2, device="cuda")
    got = M.route_experts_backward(d, x, idx, "sigmoid", False, 1.0).cpu()
    s = torch.sigmoid(x.double().cpu())[0, 3]
    assert abs(got[0, 3] - s * (1 - s)) < 1e-6 and (got[1] == 0).all()
    assert got[0].count_nonzero() == 1


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_autograd(score):
    import sparse_mixture_experts_gemv_gb300 as M
    x = _make(9, 32, "fp32", 8).requires_grad_()
    bias = torch.linspace(0, 0.1, 32, device="cuda")
    idx, w = M.route_experts(x, 4, score=score, bias=bias, groups=4, top_groups=2, scale=2.0)
    assert not idx.requires_grad and w.requires_grad
    d = torch.randn(9, 4, generator=torch.Generator().manual_seed(3)).cuda()
    w.backward(d.t().contiguous().t())      # a gradient with other strides
    ref, mag = o.route_backward(d.cpu().numpy(), x.detach().cpu().numpy(), idx.cpu().numpy(), score, True, 2.0)
    assert (np.abs(x.grad.cpu().numpy() - ref) <= REL * mag + 1e-37).all()
    with torch.no_grad():
        assert not M.route_experts(x, 4, score=score)[1].requires_grad


def test_backward_captured_in_a_graph():
    """The calls themselves (no autograd engine inside the capture) replay on new data."""
    import sparse_mixture_experts_gemv_gb300 as M
    x, d = _make(65, 128, "fp32", 4), torch.randn(65, 8, device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        M.route_experts_backward(d, x, M.route_experts(x, 8, score="sigmoid")[0], "sigmoid")
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        idx, w = M.route_experts(x, 8, score="sigmoid")
        dx = M.route_experts_backward(d, x, idx, "sigmoid")
    x.copy_(_make(65, 128, "fp32", 5))
    g.replay()
    torch.cuda.synchronize()
    i2, w2 = M.route_experts(x, 8, score="sigmoid")
    assert torch.equal(idx, i2) and torch.equal(w, w2)
    assert torch.equal(dx, M.route_experts_backward(d, x, i2, "sigmoid"))
