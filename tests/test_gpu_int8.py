"""int8_matmul and int8_experts against the fp64 oracle."""
import numpy as np
import pytest

from oracle import route_int8_oracle as o

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
STEP = 2.0 ** -24   # half a step of fp32


def _half(dtype):
    return torch.finfo(dtype).eps / 2


def _np(t):
    return t.double().cpu().numpy()


def _ints(*shape, seed=0, lo=-127, hi=128):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(lo, hi, shape, generator=g, dtype=torch.int8).cuda()


def _x(T, K, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g)
    x[:, ::97] *= 10
    return x.to(DT[dtype]).cuda()


def _scales(*shape, seed=0):
    g = torch.Generator().manual_seed(seed + 1)
    return (torch.rand(*shape, generator=g) + 0.5).cuda() * 1e-3


def _close(got, ref, rel_acc, out_dtype, mag=None):
    """Two products with scales and the sum's own conversion (3 half steps of fp32), what the
    accumulation may lose (rel_acc of the terms' magnitude), and the output's rounding."""
    tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 1e-40, torch.float32: 1e-40}[out_dtype]
    tol = 3.1 * STEP * np.abs(ref) + (0 if mag is None else rel_acc * mag) + tiny
    if out_dtype is not torch.float32:
        tol = tol + _half(out_dtype) * (np.abs(ref) + tol)
    err = np.abs(_np(got) - ref)
    assert (err <= tol).all(), (float((err / tol).max()), np.argwhere(err > tol)[:4])


SHAPES = [(1, 16, 1), (1, 2048, 1024), (2, 48, 7), (3, 256, 129), (4, 2048, 333), (5, 512, 64), (7, 80, 255),
          (8, 2560, 100), (9, 64, 128), (13, 1024, 300), (16, 128, 1), (17, 144, 127), (31, 4096, 65), (64, 512, 1000),
          (65, 336, 256), (127, 768, 129), (200, 272, 385), (333, 1040, 513), (1000, 128, 300), (1537, 2048, 160)]


@pytest.mark.parametrize("T,K,n", SHAPES)
def test_shapes(T, K, n):
    import sparse_mixture_experts_gemv_gb300 as M
    w, ws = _ints(n, K, seed=n), _scales(n, seed=n)
    q, qs = _ints(T, K, seed=T, lo=-20, hi=21), _scales(T, seed=T)
    # |sums| stay below 2^24 (20 * 127 * 4096 < 2^24): exact
    for out in DT.values():
        got = M.int8_matmul(q, w, ws, qs, out_dtype=out)
        assert got.dtype is out and got.shape == (T, n)
        _close(got, o.matmul(_np(q), _np(w), _np(ws), _np(qs)), 0, out)
    for dtype in DT:
        x = _x(T, K, dtype, seed=T)
        ref = o.matmul(_np(x), _np(w), _np(ws))
        # sums of quantized normals times bytes: sqrt(K) * 127 * 40 << 2^24 here
        _close(M.int8_matmul(x, w, ws), ref, 0, DT[dtype])
        _close(M.int8_matmul(x, w, ws, out_dtype=torch.float32), ref, 0, torch.float32)


@pytest.mark.parametrize("T,K,n", [(3, 528, 44001), (5, 272, 13201), (5, 4096, 10001), (9, 1040, 7300), (9, 4096, 5500), (17, 2064, 6001), (31, 2048, 4096), (65, 1040, 3001),
                                   (96, 1104, 2000), (193, 1552, 700), (385, 272, 2049), (1000, 336, 700),
                                   (1200, 128, 1501), (2048, 80, 1352)])
def test_shapes_on_the_tensor_cores(T, K, n):
    """Products with more results than the dot-product units take: tiles of every number of tokens, ragged in all directions."""
    import sparse_mixture_experts_gemv_gb300 as M
    w, ws = _ints(n, K, seed=n), _scales(n, seed=n)
    q, qs = _ints(T, K, seed=T, lo=-20, hi=21), _scales(T, seed=T)
    ref = o.matmul(_np(q), _np(w), _np(ws), _np(qs))
    for out in DT.values():
        _close(M.int8_matmul(q, w, ws, qs, out_dtype=out), ref, 0, out)
    for dtype in DT:
        x = _x(T, K, dtype, seed=T)
        _close(M.int8_matmul(x, w, ws, out_dtype=torch.float32), o.matmul(_np(x), _np(w), _np(ws)), 0, torch.float32)


def test_very_many_rows_of_a_tiny_product():
    import sparse_mixture_experts_gemv_gb300 as M
    T = 600000
    q, qs, w, ws = _ints(T, 16), _scales(T), _ints(3, 16), _scales(3)
    got = M.int8_matmul(q, w, ws, qs, out_dtype=torch.float32)
    _close(got, o.matmul(_np(q), _np(w), _np(ws), _np(qs)), 0, torch.float32)


def test_rows_that_are_not_finite_on_the_tensor_cores():
    import sparse_mixture_experts_gemv_gb300 as M
    w, ws = _ints(2000, 1040), _scales(2000)
    x = _x(130, 1040, "bf16")
    want = M.int8_matmul(x, w, ws)
    x[3, 5], x[77, 1039], x[129] = float("inf"), float("nan"), 0
    got = M.int8_matmul(x, w, ws)
    assert torch.isnan(got[3]).all() and torch.isnan(got[77]).all() and (got[129] == 0).all()
    others = [t for t in range(129) if t not in (3, 77)]
    assert torch.equal(got[others], want[others])


@pytest.mark.parametrize("T", [24, 40])
def test_largest_sums_on_the_tensor_cores(T):
    """As below, with sums up to 2^28 of one sign: kept to 24 bits in the accumulators."""
    import sparse_mixture_experts_gemv_gb300 as M
    K, n = 16384, 3000
    w = torch.full((n, K), 127, dtype=torch.int8)
    w[1::3] = -128
    w[2::3, ::2] = -127
    x = torch.full((T, K), -128, dtype=torch.int8)
    x[0] = 127
    ws, xs = torch.ones(n), torch.ones(T)
    got = M.int8_matmul(x.cuda(), w.cuda(), ws.cuda(), xs.cuda(), out_dtype=torch.float32)
    ref = o.matmul(_np(x), _np(w), _np(ws), _np(xs))
    mag = np.abs(_np(x)) @ np.abs(_np(w)).T
    _close(got, ref, K / 16 * 2 * STEP, torch.float32, mag)


@pytest.mark.parametrize("T", [1, 4, 20, 150])
def test_largest_sums(T):
    """All values at their largest, -128 among them: sums up to 2^27 and sums that cancel."""
    import sparse_mixture_experts_gemv_gb300 as M
    K, n = 8192, 40
    w = torch.full((n, K), 127, dtype=torch.int8)
    w[1] = -128
    w[2, ::2] = -127
    w[3, : K // 2] = -128
    x = torch.full((T, K), -128, dtype=torch.int8)
    x[0] = 127
    ws, xs = torch.ones(n), torch.ones(T)
    got = M.int8_matmul(x.cuda(), w.cuda(), ws.cuda(), xs.cuda(), out_dtype=torch.float32)
    ref = o.matmul(_np(x), _np(w), _np(ws), _np(xs))
    mag = np.abs(_np(x)) @ np.abs(_np(w)).T
    # 512 accumulations of 16 products, each sum kept to 24 bits
    _close(got, ref, K / 16 * 2 * STEP, torch.float32, mag)


@pytest.mark.parametrize("T", [1, 6, 40, 260])
def test_rows_of_zeros_infinities_and_ties(T):
    import sparse_mixture_experts_gemv_gb300 as M
    K, n = 256, 48
    w, ws = _ints(n, K), _scales(n)
    for dtype in DT:
        x = _x(T, K, dtype)
        x[T - 1] = 0
        got = M.int8_matmul(x, w, ws, out_dtype=torch.float32)
        assert (got[T - 1] == 0).all()
        # halves of the largest value are ties but for the scale's rounding; exact ties go to even
        y = x.clone()
        y[0] = torch.linspace(-1, 1, K).to(DT[dtype]).cuda()
        y[0, ::2] = torch.arange(K // 2, device="cuda").to(DT[dtype]) % 64 + 0.5
        y[0, 1] = 127
        y[T - 1] = 3.0
        y[T - 1, ::2] = 1.5
        _close(M.int8_matmul(y, w, ws, out_dtype=torch.float32), o.matmul(_np(y), _np(w), _np(ws)), 0, torch.float32)
        for bad in (float("inf"), -float("inf"), float("nan")):
            z = x.clone()
            z[0, 5] = bad
            got = M.int8_matmul(z, w, ws, out_dtype=torch.float32)
            assert torch.isnan(got[0]).all()
            assert T == 1 or torch.isfinite(got[1:]).all()


@pytest.mark.parametrize("T", [2, 30])
@pytest.mark.parametrize("size", [1e-44, 3e-39, 1e-33, 1e-28, 1e25, 3e38])
def test_extreme_magnitudes(T, size):
    import sparse_mixture_experts_gemv_gb300 as M
    x = torch.randn(T, 128, generator=torch.Generator().manual_seed(1)).clamp(-1, 1)
    x[:, 0] = 1.0
    x = (x.double() * size).float().cuda()
    w, ws = _ints(32, 128), torch.ones(32, device="cuda")
    got = _np(M.int8_matmul(x, w, ws, out_dtype=torch.float32))
    q, s, near = o.quantize(_np(x))
    # results below the normal range round to steps of 2^-149, three times
    ref = o.matmul(_np(x), _np(w), _np(ws))
    tol = 3.1 * STEP * np.abs(ref) + 3 * 2.0 ** -149
    ok = np.abs(ref) < 3.4e38
    assert (np.abs(got - ref)[ok] <= tol[ok]).all()
    assert not np.isfinite(got[~ok]).any()


def test_strides_alignment_and_defaults():
    import sparse_mixture_experts_gemv_gb300 as M
    base, wb = _x(300, 320, "bf16"), _ints(200, 272)
    ws = _scales(200)
    big, big_ws = _ints(3000, 272, seed=3), _scales(3000, seed=3)
    for x, w in ((base[:, :256], big[:, :256]), (base[:, 8:264], big[:, 16:]), (base[:, 3:259], big[:, 5:261])):
        _close(M.int8_matmul(x, w, big_ws), o.matmul(_np(x), _np(w), _np(big_ws)), 0, torch.bfloat16)
    for T in (3, 300):
        for x, w in ((base[:T, :256], wb[:, :256]), (base[:T, 8:264], wb[:, 16:]), (base[:T, 3:259], wb[:, 5:261]),
                     (base[:T, :256].t().contiguous().t(), wb[:, :256]), (base[:, :256][:2 * T:2], wb[:, :256])):
            got = M.int8_matmul(x, w, ws)
            assert got.dtype is torch.bfloat16
            _close(got, o.matmul(_np(x), _np(w), _np(ws)), 0, torch.bfloat16)
    q, qs = _ints(300, 320, lo=-30, hi=31), _scales(300)
    got = M.int8_matmul(q[:, 32:288], wb[:, :256], _scales(400)[::2], qs)
    assert got.dtype is torch.bfloat16
    _close(got, o.matmul(_np(q[:, 32:288]), _np(wb[:, :256]), _np(_scales(400)[::2]), _np(qs)), 0, torch.bfloat16)
    for T, n in ((0, 5), (5, 0)):
        assert M.int8_matmul(base[:T, :256], wb[:n, :256], ws[:n]).shape == (T, n)


def test_refusals():
    import sparse_mixture_experts_gemv_gb300 as M
    x, w, ws = _x(4, 64, "bf16"), _ints(8, 64), _scales(8)
    for bad in (lambda: M.int8_matmul(x, w[:, :48], ws), lambda: M.int8_matmul(x, w.float(), ws),
                lambda: M.int8_matmul(x, w, ws[:7]), lambda: M.int8_matmul(x, w, ws.double()),
                lambda: M.int8_matmul(x, w, ws, torch.ones(4, device="cuda")), lambda: M.int8_matmul(w, w, ws),
                lambda: M.int8_matmul(x, w, ws, out_dtype=torch.int8), lambda: M.int8_matmul(x, w.cpu(), ws),
                lambda: M.int8_matmul(x.double(), w, ws), lambda: M.int8_matmul(x[0], w, ws)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises((ValueError, M.MoeError)):
        M.int8_matmul(x[:, :40], w[:, :40], ws)   # K = 40


def test_streams_graph_and_repeats():
    import sparse_mixture_experts_gemv_gb300 as M
    w, ws = _ints(1777, 512), _scales(1777)
    for T in (1, 8, 300):
        x = _x(T, 512, "bf16")
        want = M.int8_matmul(x, w, ws)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        got = [M.int8_matmul(x, w, ws, stream=s) for _ in range(4)]
        s.synchronize()
        assert all(torch.equal(want, a) for a in got)
        g = torch.cuda.CUDAGraph()
        y = x.clone()
        with torch.cuda.graph(g):
            out = M.int8_matmul(y, w, ws)
        y.copy_(_x(T, 512, "bf16", seed=5))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, M.int8_matmul(y, w, ws))


# ------------------------------------------------------------------------------------------- experts
def _experts(E, H, I, seed=0):
    return (_ints(E, 2 * I, H, seed=seed), _scales(E, 2 * I, seed=seed) / 30, _ints(E, H, I, seed=seed + 1),
            _scales(E, H, seed=seed + 1))


def _choices(T, E, k, seed=0):
    g = torch.Generator().manual_seed(seed)
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]) if T else torch.empty(0, k)
    return idx.to(torch.int32).cuda(), torch.softmax(torch.randn(T, k, generator=g), 1).cuda()


def _check_experts(x, idx, w, ex, got):
    ref, mag, unsure = o.experts(_np(x), idx.cpu().numpy(), _np(w), *(_np(a) for a in ex))
    # the products' and scales' roundings, exp and the quotient of SwiGLU, sums over I and k: 2^-17 of
    # the terms' magnitude; integer sums kept in 16 bits on the way to the weighted sum: 2^-11 of each
    # term's own size, not of its parts', which half of the type's step below covers k times over
    tol = 2.0 ** -17 * mag + unsure
    tol = tol + 1.5 * _half(x.dtype) * (np.abs(ref) + tol) + 2.0 ** -11 * _term_sizes(x, idx, w, ex) + 2.0 ** -24
    err = np.abs(_np(got) - ref)
    assert (err <= tol).all(), (float((err / tol).max()), np.argwhere(err > tol)[:4])


def _term_sizes(x, idx, w, ex):
    """sum_j |weights[t, j] y_j[t]|, one choice at a time."""
    total = 0.0
    for j in range(idx.shape[1]):
        one, _, _ = o.experts(_np(x), idx[:, j:j + 1].cpu().numpy(), _np(w)[:, j:j + 1], *(_np(a) for a in ex))
        total = total + np.abs(one)
    return total


@pytest.mark.parametrize("T,E,k,H,I", [(1, 1, 1, 16, 16), (1, 16, 8, 256, 128), (2, 5, 2, 48, 80), (4, 64, 8, 512, 96),
                                       (5, 16, 4, 272, 64), (8, 256, 8, 128, 32), (9, 8, 3, 256, 144), (17, 4, 4, 128, 64),
                                       (33, 16, 1, 336, 112), (64, 60, 6, 256, 128), (130, 16, 8, 640, 192),
                                       (300, 3, 2, 128, 64), (513, 32, 8, 128, 48)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_experts(T, E, k, H, I, dtype):
    import sparse_mixture_experts_gemv_gb300 as M
    x, (idx, w), ex = _x(T, H, dtype, seed=T), _choices(T, E, k, seed=E), _experts(E, H, I, seed=H)
    got = M.int8_experts(x, idx, w, *ex)
    assert got.dtype is x.dtype and got.shape == x.shape
    _check_experts(x, idx, w, ex, got)


def test_more_choices_than_are_counted_at_once():
    """T * k above 32,768: sampled tokens against the same tokens in a call of their own."""
    import sparse_mixture_experts_gemv_gb300 as M
    T, E, k, H, I = 4500, 20, 8, 64, 32
    x, (idx, w), ex = _x(T, H, "bf16"), _choices(T, E, k), _experts(E, H, I)
    idx[5] = -1
    got = M.int8_experts(x, idx, w, *ex)
    some = torch.tensor([0, 1, 5, 31, 32, 2222, 4463, 4464, 4499], device="cuda")
    assert (got[5] == 0).all()
    _check_experts(x[some], idx[some], w[some], ex, got[some])


@pytest.mark.parametrize("T", [3, 100])
def test_choices_left_out_and_uneven_loads(T):
    import sparse_mixture_experts_gemv_gb300 as M
    E, k, H, I = 24, 4, 256, 64
    x, (idx, w), ex = _x(T, H, "bf16"), _choices(T, E, k), _experts(E, H, I)
    idx[0] = -1                      # a row with no choice
    idx[1, 2] = E                    # out of range
    idx[1, 0] = 2 ** 31 - 1
    idx[2:, 0] = 7                   # one expert for nearly all tokens
    idx[2:, 1:] = torch.where(idx[2:, 1:] == 7, -1, idx[2:, 1:])
    got = M.int8_experts(x, idx, w, *ex)
    assert (got[0] == 0).all()
    _check_experts(x, idx, w, ex, got)
    none = M.int8_experts(x, torch.full_like(idx, -5), w, *ex)
    assert (none == 0).all()
    assert M.int8_experts(x[:0], idx[:0], w[:0], *ex).shape == (0, H)


@pytest.mark.parametrize("T", [2, 70])
def test_rows_that_are_not_finite_stay_alone(T):
    import sparse_mixture_experts_gemv_gb300 as M
    x, (idx, w), ex = _x(T, 128, "bf16"), _choices(T, 8, 2), _experts(8, 128, 32)
    want = M.int8_experts(x, idx, w, *ex)
    x[1, 3] = float("inf")
    got = M.int8_experts(x, idx, w, *ex)
    assert torch.isnan(got[1]).all() and torch.equal(got[0], want[0])
    assert T == 2 or torch.equal(got[2:], want[2:])
    x[1] = 0
    assert (M.int8_experts(x, idx, w, *ex)[1] == 0).all()


@pytest.mark.parametrize("T", [1, 6, 90])
def test_experts_streams_graph_and_repeats(T):
    import sparse_mixture_experts_gemv_gb300 as M
    x, (idx, w), ex = _x(T, 256, "bf16"), _choices(T, 32, 4), _experts(32, 256, 64)
    want = M.int8_experts(x, idx, w, *ex)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = [M.int8_experts(x, idx, w, *ex, stream=s) for _ in range(4)]
    s.synchronize()
    assert all(torch.equal(want, a) for a in got)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = M.int8_experts(x, idx, w, *ex)
    i2, w2 = _choices(T, 32, 4, seed=9)
    idx.copy_(i2)
    w.copy_(w2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, M.int8_experts(x, idx, w, *ex))


def test_experts_refusals():
    import sparse_mixture_experts_gemv_gb300 as M
    x, (idx, w), ex = _x(4, 64, "bf16"), _choices(4, 8, 2), _experts(8, 64, 32)
    gu, gus, dn, dns = ex
    for args in ((x.float(), idx, w, *ex), (x, idx.long(), w, *ex), (x, idx[:3], w, *ex), (x, idx, w.half(), *ex),
                 (x, idx, w, gu[:, :31], gus, dn, dns), (x, idx, w, gu, gus[:, :5], dn, dns),
                 (x, idx, w, gu, gus, dn[:, :, :16], dns), (x, idx, w, gu, gus, dn, dns.cpu()),
                 (x, idx, w, gu.transpose(0, 1), gus, dn, dns), (x[:, :48], idx, w, *ex)):
        with pytest.raises(ValueError):
            M.int8_experts(*args)
