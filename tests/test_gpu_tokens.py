"""dispatch_tokens and combine_tokens against the fp64 oracle: types, odd sizes, choices of no expert, strides, both
sides of the choice between one launch and two, gradients, refusals.

A copied value is the same bits. A sum of k products in fp32 is off by at most k roundings of its terms' magnitudes
(each addition with its product is one fma, 2^-24 of at most that sum), a dot product of H terms by H of them, and the
result's own rounding by eps / 2 of it."""
import numpy as np
import pytest

from oracle import tokens_fp8_oracle as o

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _idx(T, k, E, seed=0, off=0.1):
    """Choices with repeats in a row, some outside [0, E)."""
    g = _gen(seed)
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    wrong = torch.tensor([-1, E, -2 ** 31, 2 ** 31 - 1], dtype=torch.int64, device="cuda").to(torch.int32)
    bad = torch.rand(T, k, generator=g, device="cuda") < off
    return torch.where(bad, wrong[torch.randint(0, 4, (T, k), generator=g, device="cuda")], idx)


def _np(t):
    return t.detach().double().cpu().numpy()


def _bytes(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def _check_dispatch(x, idx, E, got):
    rows, offsets, pos = got
    want_offsets, want_pos = o.places(idx.cpu().numpy(), E)
    np.testing.assert_array_equal(offsets.cpu().numpy(), want_offsets)
    np.testing.assert_array_equal(pos.cpu().numpy(), want_pos)
    np.testing.assert_array_equal(_bytes(rows), o.dispatch(_bytes(x), want_pos))


# (T, k, E, H): up to 2,048 choices every CTA places all, in one segment of 512 and in several; up to 32,768 it counts
# all and places its chunk; beyond, a launch counts. Chunks of more than 1,024 choices have several segments.
SHAPES = [(1, 8, 256, 2048), (1, 1, 1, 1), (3, 2, 5, 7), (64, 8, 16, 33), (65, 8, 1024, 130), (256, 8, 64, 24),
          (257, 8, 64, 24), (2049, 1, 1, 5), (70, 32, 3, 260), (1000, 7, 1023, 96), (5000, 3, 511, 9),
          (4096, 8, 256, 16), (4097, 8, 256, 16), (9000, 32, 1024, 4), (6007, 31, 40, 3)]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,k,E,H", SHAPES)
def test_dispatch(T, k, E, H, dtype):
    import sparse_mixture_experts_gemv_gb300 as M
    x = torch.randn(T, H, generator=_gen(1), device="cuda").to(DT[dtype])
    idx = _idx(T, k, E)
    got = M.dispatch_tokens(x, idx, E)
    _check_dispatch(x, idx, E, got)
    again = M.dispatch_tokens(x, idx, E)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("off", [0.0, 1.0])
@pytest.mark.parametrize("T", [5, 700])
def test_dispatch_of_all_or_no_choices(T, off):
    import sparse_mixture_experts_gemv_gb300 as M
    x = torch.randn(T, 40, generator=_gen(1), device="cuda").bfloat16()
    idx = _idx(T, 4, 9, off=off)
    _check_dispatch(x, idx, 9, M.dispatch_tokens(x, idx, 9))


@pytest.mark.parametrize("T", [0, 1, 300, 3000])
def test_dispatch_of_quantized_rows_takes_their_scales_along(T):
    import sparse_mixture_experts_gemv_gb300 as M
    for dtype, H, n in ((torch.float8_e4m3fn, 528, 5), (torch.uint8, 37, 1), (torch.int8, 128, 40)):
        x = torch.randint(0, 127, (T, H), generator=_gen(3), device="cuda").to(torch.uint8).view(dtype)
        scale = torch.rand(T, n, generator=_gen(4), device="cuda")
        idx = _idx(T, 3, 17)
        rows, row_scale, offsets, pos = M.dispatch_tokens(x, idx, 17, scale)
        assert rows.dtype is dtype and rows.shape == (3 * T, H) and row_scale.shape == (3 * T, n)
        _check_dispatch(x.view(torch.uint8), idx, 17, (rows.view(torch.uint8), offsets, pos))
        np.testing.assert_array_equal(row_scale.cpu().numpy(), o.dispatch(scale.cpu().numpy(), o.places(idx.cpu().numpy(), 17)[1]))


def test_dispatch_of_rows_apart_and_off_their_boundaries():
    """Every vector width: rows of 16, 8, 4, 2 and 1 bytes' alignment, apart, transposed and repeated."""
    import sparse_mixture_experts_gemv_gb300 as M
    wide = torch.randn(50, 300, generator=_gen(5), device="cuda").bfloat16()
    idx = _idx(50, 4, 6)
    for x in (wide[:, :256], wide[:, 8:264], wide[:, 4:260], wide[:, 2:258], wide[:, 1:258], wide[:, 1:2], wide.T[:50, :50],
              wide[:1, 3:].expand(50, 297), wide[:, ::2]):
        _check_dispatch(x, idx, 6, M.dispatch_tokens(x, idx, 6))
    one = wide.as_strided((1, 64), (3, 1), 5)
    _check_dispatch(one, idx[:1], 6, M.dispatch_tokens(one, idx[:1], 6))
    turned = idx.T.contiguous().T
    _check_dispatch(wide, turned, 6, M.dispatch_tokens(wide, turned, 6))
    b = wide.view(torch.uint8)[:, 3:200]
    _check_dispatch(b, idx, 6, M.dispatch_tokens(b, idx, 6))


@pytest.mark.parametrize("T", [100, 3000, 20000])
def test_choices_off_their_boundaries(T):
    """A view whose first choice lies off a 16-byte boundary."""
    import sparse_mixture_experts_gemv_gb300 as M
    x = torch.randn(T, 12, generator=_gen(1), device="cuda")
    idx = _idx(T + 1, 3, 40)[1:]
    assert idx.is_contiguous() and idx.data_ptr() % 16
    _check_dispatch(x, idx, 40, M.dispatch_tokens(x, idx, 40))


def test_dispatch_of_no_tokens():
    import sparse_mixture_experts_gemv_gb300 as M
    rows, offsets, pos = M.dispatch_tokens(torch.empty(0, 16, device="cuda"), torch.empty(0, 4, dtype=torch.int32, device="cuda"), 700)
    assert rows.shape == (0, 16) and pos.shape == (0, 4) and offsets.tolist() == [0] * 701
    assert M.dispatch_tokens_backward(rows, pos).shape == (0, 16)
    w = torch.empty(0, 4, device="cuda")
    assert M.combine_tokens(rows, pos, w).shape == (0, 16)
    d_y, d_w = M.combine_tokens_backward(torch.empty(0, 16, device="cuda"), rows, pos, w)
    assert d_y.shape == (0, 16) and d_w.shape == (0, 4)


def _combine_inputs(T, k, E, H, dtype, off=0.1, scale=1.0):
    pos = torch.from_numpy(o.places(_idx(T, k, E, 7, off).cpu().numpy(), E)[1].astype(np.int32)).cuda()
    y = (scale * torch.randn(T * k, H, generator=_gen(8), device="cuda")).to(DT[dtype])
    w = torch.randn(T, k, generator=_gen(9), device="cuda")
    d = torch.randn(T, H, generator=_gen(10), device="cuda").to(DT[dtype])
    return y, pos, w, d


def _near(got, want, mag, terms, dtype):
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps   # half a step below the normal range, and the sum's own there
    bound = np.abs(want) * half * (1 + 2 ** -20) + terms * 2.0 ** -24 * 1.01 * mag + tiny
    bad = np.abs(_np(got) - want) > bound
    assert not bad.any(), (np.argwhere(bad)[:5], _np(got)[bad][:5], want[bad][:5])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,k,E,H", [(1, 8, 64, 2048), (4, 8, 512, 2560), (3, 1, 4, 1), (33, 7, 9, 257), (130, 32, 11, 72),
                                     (900, 9, 40, 96), (5000, 2, 8, 8)])
def test_combine_and_its_gradients(T, k, E, H, dtype):
    import sparse_mixture_experts_gemv_gb300 as M
    y, pos, w, d = _combine_inputs(T, k, E, H, dtype)
    p = pos.cpu().numpy()
    want, mag = o.combine(_np(y), p, _np(w))
    _near(M.combine_tokens(y, pos, w), want, mag, k, DT[dtype])
    d_y, d_w = M.combine_tokens_backward(d, y, pos, w)
    want_y, want_w, mag = o.combine_backward(_np(d), _np(y), p, _np(w))
    _near(d_y, want_y, np.abs(want_y), 1, DT[dtype])
    _near(d_w, want_w, mag, H, torch.float32)
    want, mag = o.combine(_np(y), p, np.ones((T, k)))
    _near(M.dispatch_tokens_backward(y, pos), want, mag, k, DT[dtype])
    assert torch.equal(M.combine_tokens_backward(d, y, pos, w)[1], d_w)   # the same bits each time


@pytest.mark.parametrize("off", [0.0, 1.0])
def test_combine_of_all_or_no_choices(off):
    import sparse_mixture_experts_gemv_gb300 as M
    y, pos, w, d = _combine_inputs(20, 3, 5, 64, "bf16", off)
    p = pos.cpu().numpy()
    want, mag = o.combine(_np(y), p, _np(w))
    _near(M.combine_tokens(y, pos, w), want, mag, 3, torch.bfloat16)
    d_y, d_w = M.combine_tokens_backward(d, y, pos, w)
    want_y, want_w, mag = o.combine_backward(_np(d), _np(y), p, _np(w))
    _near(d_y, want_y, np.abs(want_y), 1, torch.bfloat16)
    _near(d_w, want_w, mag, 64, torch.float32)


def test_rows_of_no_expert_are_not_read():
    """Infinities and NaN in rows that no choice has a place in, and in d_out's weights that are off."""
    import sparse_mixture_experts_gemv_gb300 as M
    y, pos, w, d = _combine_inputs(40, 4, 6, 128, "fp32", 0.3)
    off = pos < 0
    clean = [M.combine_tokens(y, pos, w), *M.combine_tokens_backward(d, y, pos, w), M.dispatch_tokens_backward(y, pos)]
    y = y.clone()
    y[(~pos[off]).long()] = float("nan")
    w = torch.where(off, float("inf"), w)
    for a, b in zip(clean, [M.combine_tokens(y, pos, w), *M.combine_tokens_backward(d, y, pos, w), M.dispatch_tokens_backward(y, pos)]):
        assert torch.equal(a, b)
    assert not clean[1][(~pos[off]).long()].any() and not clean[2][off].any()


def test_places_outside_the_rows_add_nothing():
    import sparse_mixture_experts_gemv_gb300 as M
    y, pos, w, d = _combine_inputs(10, 4, 6, 64, "fp32", 0.0)
    wrong = pos.clone()
    wrong[0, 0], wrong[1, 1], wrong[2, 2], wrong[3, 3] = 40, 2 ** 31 - 1, -2 ** 31, -41
    none = (wrong >= 40) | (wrong < 0)
    want, mag = o.combine(_np(y), np.where(none.cpu().numpy(), -1, pos.cpu().numpy()), _np(w))
    _near(M.combine_tokens(y, wrong, w), want, mag, 4, torch.float32)
    d_y, d_w = M.combine_tokens_backward(d, y, wrong, w)
    assert not d_w[none].any()
    keep = pos[~none].long()
    assert torch.equal(d_y[keep], M.combine_tokens_backward(d, y, pos, w)[0][keep])


def test_infinite_and_nan_rows_stay_with_their_tokens():
    import sparse_mixture_experts_gemv_gb300 as M
    y, pos, w, _ = _combine_inputs(9, 2, 3, 64, "bf16", 0.0)
    y[pos[4, 1].long(), 7], y[pos[5, 0].long(), 9] = float("inf"), float("nan")
    out = M.combine_tokens(y, pos, w)
    bad = ~out.isfinite()
    assert bad[4, 7] and out[5, 9].isnan() and int(bad.sum()) == 2


def test_combine_of_rows_apart():
    import sparse_mixture_experts_gemv_gb300 as M
    y, pos, w, d = _combine_inputs(30, 3, 5, 64, "bf16")
    want = [M.combine_tokens(y, pos, w), *M.combine_tokens_backward(d, y, pos, w), M.dispatch_tokens_backward(y, pos)]
    for pad in (8, 3):
        ya = torch.zeros(90, 64 + 2 * pad, dtype=y.dtype, device="cuda")[:, pad:64 + pad].copy_(y)
        da = torch.zeros(30, 64 + pad, dtype=y.dtype, device="cuda")[:, pad:].copy_(d)
        got = [M.combine_tokens(ya, pos, w), *M.combine_tokens_backward(da, ya, pos, w), M.dispatch_tokens_backward(ya, pos)]
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[3], want[3])
        # another width adds the products of a row in another order
        assert torch.allclose(got[2], want[2], rtol=0, atol=64 * 2.0 ** -24 * float((d.float().abs().max() * y.float().abs().max()) * 64))
    one = d[:1].expand(30, 64)
    got = M.combine_tokens_backward(one, y, pos, w)
    again = M.combine_tokens_backward(one.contiguous(), y, pos.T.contiguous().T, w.T.contiguous().T)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_gradients_through_the_graph_and_against_differences():
    import sparse_mixture_experts_gemv_gb300 as M
    T, k, E, H = 12, 3, 5, 32
    idx = _idx(T, k, E, 11, 0.2)
    x = torch.randn(T, H, generator=_gen(12), device="cuda", requires_grad=True)
    w = torch.rand(T, k, generator=_gen(13), device="cuda", requires_grad=True)
    mix = torch.randn(T, H, generator=_gen(14), device="cuda")

    def loss(x, w):
        rows, offsets, pos = M.dispatch_tokens(x, idx, E)
        assert not offsets.requires_grad and not pos.requires_grad
        return (M.combine_tokens(rows * rows, pos, w) * mix).sum()

    gx, gw = torch.autograd.grad(loss(x, w), (x, w))
    on = ((idx >= 0) & (idx < E)).double()
    # the same function, written out
    xd, wd, md = x.detach().double(), w.detach().double(), mix.double()
    want_x = 2 * xd * md * (wd * on).sum(1, keepdim=True)
    want_w = (xd * xd * md).sum(1, keepdim=True) * on
    assert torch.allclose(gx.double(), want_x, rtol=1e-5, atol=1e-5)
    assert torch.allclose(gw.double(), want_w, rtol=1e-5, atol=1e-4)

    def value(x, w):
        return float(((x * x) * (w * on).sum(1, keepdim=True) * md).sum())
    dx, dw = torch.randn_like(x).double(), torch.randn_like(w).double()
    h = 1e-5
    diff = (value(xd + h * dx, wd + h * dw) - value(xd - h * dx, wd - h * dw)) / (2 * h)
    got = float((gx * dx).sum() + (gw * dw).sum())
    assert abs(got - diff) < 1e-4 * float((gx * dx).abs().sum() + (gw * dw).abs().sum())
    # one of the two alone
    assert torch.equal(torch.autograd.grad(loss(x, w.detach()), x)[0], gx)
    assert torch.equal(torch.autograd.grad(loss(x.detach(), w), w)[0], gw)
    assert not loss(x.detach(), w.detach()).requires_grad


def test_second_derivatives_are_refused():
    import sparse_mixture_experts_gemv_gb300 as M
    idx = _idx(6, 2, 4, off=0.0)
    x = torch.randn(6, 16, device="cuda", requires_grad=True)
    w = torch.rand(6, 2, device="cuda", requires_grad=True)
    rows, _, pos = M.dispatch_tokens(x, idx, 4)
    out = M.combine_tokens(rows, pos, w)
    g, = torch.autograd.grad(out.square().sum(), w, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        g.sum().backward()
    d = torch.ones(12, 16, device="cuda", requires_grad=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        M.dispatch_tokens_backward(d, pos).sum().backward()
    with pytest.raises(RuntimeError, match="second derivative"):
        M.combine_tokens_backward(torch.ones(6, 16, device="cuda"), rows, pos, w)[0].sum().backward()


def test_on_another_stream_and_captured():
    """A captured forward and backward, replayed on new inputs, beside an eager call's."""
    import sparse_mixture_experts_gemv_gb300 as M
    T, k, E, H = 400, 8, 32, 256
    idx, x = _idx(T, k, E, 20), torch.randn(T, H, generator=_gen(21), device="cuda").bfloat16()
    w = torch.rand(T, k, generator=_gen(22), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    want = M.dispatch_tokens(x, idx, E)
    got = M.dispatch_tokens(x, idx, E, stream=s)
    out = M.combine_tokens(got[0], got[2], w, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert torch.equal(out, M.combine_tokens(want[0], want[2], w))

    def step():
        rows, offsets, pos = M.dispatch_tokens(x, idx, E)
        out = M.combine_tokens(rows, pos, w)
        return (rows, offsets, pos, out, *M.combine_tokens_backward(out, rows, pos, w), M.dispatch_tokens_backward(rows, pos))

    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        held = step()
    for seed in (30, 31):
        idx.copy_(_idx(T, k, E, seed))
        x.copy_(torch.randn(T, H, generator=_gen(seed), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, step()))


def test_refusals():
    import sparse_mixture_experts_gemv_gb300 as M
    x, idx = torch.randn(4, 16, device="cuda"), _idx(4, 2, 3, off=0.0)
    rows, offsets, pos = M.dispatch_tokens(x, idx, 3)
    w = torch.rand(4, 2, device="cuda")
    for call in (lambda: M.dispatch_tokens(x.double(), idx, 3), lambda: M.dispatch_tokens(x[0], idx, 3),
                 lambda: M.dispatch_tokens(x, idx.long(), 3), lambda: M.dispatch_tokens(x, idx[:3], 3),
                 lambda: M.dispatch_tokens(x, idx.cpu(), 3), lambda: M.dispatch_tokens(x, idx, 0),
                 lambda: M.dispatch_tokens(x, idx, torch.tensor(3)), lambda: M.dispatch_tokens(x, idx[:, :0], 3),
                 lambda: M.dispatch_tokens(x[:, :0], idx, 3), lambda: M.dispatch_tokens(x, idx, 3, w[:3]),
                 lambda: M.dispatch_tokens(x, idx, 3, w.double()), lambda: M.dispatch_tokens(x, idx, 3, w[:, :0]),
                 lambda: M.combine_tokens(rows, pos, w.half()), lambda: M.combine_tokens(rows, pos, w[:, :1]),
                 lambda: M.combine_tokens(rows[:7], pos, w), lambda: M.combine_tokens(rows, pos.long(), w),
                 lambda: M.combine_tokens(rows.double(), pos, w), lambda: M.combine_tokens(rows, pos, w.cpu()),
                 lambda: M.combine_tokens(rows, pos, None), lambda: M.dispatch_tokens_backward(rows[:5], pos),
                 lambda: M.combine_tokens_backward(x.half(), rows, pos, w), lambda: M.combine_tokens_backward(x[:3], rows, pos, w),
                 lambda: M.combine_tokens_backward(x, rows, pos, None)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: M.dispatch_tokens(x, idx, 1025), lambda: M.dispatch_tokens(x, idx.repeat(1, 17), 3)):
        with pytest.raises(M.MoeError):
            call()
