"""What the gradient of route_experts does at its edges: values that are not finite come through, and derivatives
that there are none of are refused and not left out."""
import pytest

from test_gpu_route_experts import DT, _make

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("E", [64, 33])      # rows in 16-byte pieces, and not
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_gradients_that_are_not_finite_come_through(dtype, E, score, renormalise):
    import sparse_mixture_experts_gemv_gb300 as M
    x = _make(6, E, dtype, 3)
    idx, _ = M.route_experts(x, 4, score=score, renormalise=renormalise)
    d = torch.randn(6, 4, generator=torch.Generator().manual_seed(1)).cuda()
    want = M.route_experts_backward(d, x, idx, score, renormalise)
    d[1, 2], d[4, 0], d[5, 3] = NAN, INF, -INF
    got = M.route_experts_backward(d, x, idx, score, renormalise)
    assert torch.equal(got[[0, 2, 3]], want[[0, 2, 3]])
    # with a sum over the row's gradients all of its chosen take the value on, else the one alone
    sums = renormalise or score == "softmax"
    for t, j in ((1, 2), (4, 0), (5, 3)):
        at = idx[t].long() if sums else idx[t, j:j + 1].long()
        assert not torch.isfinite(got[t, at]).any(), (t, got[t, at])
        assert torch.isnan(got[t, idx[t, j].long()]) == (sums or t == 1)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("E", [64, 33])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_experts_that_are_off_have_no_gradient_whatever_the_others_have(dtype, E, score, renormalise):
    import sparse_mixture_experts_gemv_gb300 as M
    x = _make(4, E, dtype, 5)
    x[:, ::3] = -INF
    x[2, 1] = NAN
    x[3, 2:] = -INF                  # fewer on than chosen
    idx, _ = M.route_experts(x, 4, score=score, renormalise=renormalise)
    d = torch.randn(4, 4, generator=torch.Generator().manual_seed(1)).cuda()
    d[0, 1], d[1, 0], d[2, 2], d[3, 0] = NAN, INF, NAN, NAN
    got = M.route_experts_backward(d, x, idx, score, renormalise)
    off = torch.isnan(x) | (x == -INF)
    assert (got[off] == 0).all()
    assert not torch.isfinite(got[~off]).all()


def test_a_second_derivative_is_refused():
    import sparse_mixture_experts_gemv_gb300 as M
    for loss in (lambda w: (w * w).sum(), lambda w: w[:, 0].sum()):     # gradients that depend on w, and do not
        x = _make(5, 16, "fp32", 2).requires_grad_()
        _, w = M.route_experts(x, 3, score="sigmoid")
        g, = torch.autograd.grad(loss(w), x, create_graph=True)
        assert g.requires_grad
        with pytest.raises(RuntimeError, match="second derivative"):
            ((g * g).sum() + (x * x).sum()).backward()
    x = _make(5, 16, "fp32", 2).requires_grad_()
    _, w = M.route_experts(x, 3, score="sigmoid")
    want, = torch.autograd.grad((w * w).sum(), x, retain_graph=True)
    got, = torch.autograd.grad((w * w).sum(), x, create_graph=True)
    assert torch.equal(want, got.detach()) and not want.requires_grad


def test_the_gradients_own_call_is_refused_the_same_way():
    import sparse_mixture_experts_gemv_gb300 as M
    x, d = _make(5, 16, "fp32", 2), torch.ones(5, 3, device="cuda")
    idx, _ = M.route_experts(x, 3)
    want = M.route_experts_backward(d, x, idx)
    assert not want.requires_grad
    for a, b in ((x.clone().requires_grad_(), d), (x, d.clone().requires_grad_())):
        got = M.route_experts_backward(b, a, idx)
        assert torch.equal(got.detach(), want)
        with pytest.raises(RuntimeError, match="second derivative"):
            got.sum().backward()
        with torch.no_grad():
            assert not M.route_experts_backward(b, a, idx).requires_grad


def test_tangents_are_refused():
    import sparse_mixture_experts_gemv_gb300 as M
    from torch.autograd import forward_ad
    x, d = _make(5, 16, "fp32", 2), torch.ones(5, 3, device="cuda")
    idx, w = M.route_experts(x, 3)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        with pytest.raises(ValueError, match="tangent"):
            M.route_experts(dual, 3)
        with pytest.raises(ValueError, match="tangent"):
            M.route_experts_backward(d, dual, idx)
        assert torch.equal(M.route_experts(x, 3)[1], w)      # without one all is as ever
