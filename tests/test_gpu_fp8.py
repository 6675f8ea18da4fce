"""fp8_quantize, fp8_matmul and fp8_grouped_matmul against the fp64 oracle.

Quantized values and scales are the oracle's bit for bit (both hold scale and quotient in 32 bits); with a SwiGLU in
front, whose 32-bit value is off by a few 2^-24 of itself, a scale is off by as much and a value by one step at most.
A product: a block's 128 terms are added up by the tensor cores in fp32 in some order, each addition off by at most
2^-23 of its operands' magnitudes whether it rounds or cuts, and so are the sums of the blocks with their scales
(fp32, 2^-24): (128 + blocks + 2) 2^-23 of the terms' magnitudes in all, and eps / 2 of the result when it is stored."""
import numpy as np
import pytest

from oracle import tokens_fp8_oracle as o

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
F8 = torch.float8_e4m3fn


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _np(t):
    return t.double().cpu().numpy()


def _codes(t):
    return t.view(torch.uint8).cpu().numpy()


def _x(T, K, dtype, seed=1):
    x = torch.randn(T, K, generator=_gen(seed), device="cuda")
    x = x * (1 + 9 * (torch.rand(K, generator=_gen(seed + 1), device="cuda") < 0.05))
    return x.to(DT[dtype])


def _w(*shape, seed=2):
    """Weights of all magnitudes that E4M3 has, and block scales over three powers of ten."""
    w = (torch.randn(*shape, generator=_gen(seed), device="cuda") * 120).clamp(-448, 448).to(F8)
    n, K = -(-shape[-2] // 128), -(-shape[-1] // 128)
    s = 10 ** (3 * torch.rand(*shape[:-2], n, K, generator=_gen(seed + 1), device="cuda") - 4)
    return w, s


def _q(T, K, seed=3):
    q = (torch.randn(T, K, generator=_gen(seed), device="cuda") * 100).clamp(-448, 448).to(F8)
    return q, torch.rand(T, -(-K // 128), generator=_gen(seed + 1), device="cuda") + 0.01


def _near(got, want, mag, K, dtype):
    blocks = -(-K // 128)
    half = torch.finfo(DT[dtype]).eps / 2
    tiny = torch.finfo(DT[dtype]).smallest_normal * torch.finfo(DT[dtype]).eps
    bound = np.abs(want) * half + (128 + blocks + 2) * 2.0 ** -23 * mag * (1 + half) + tiny
    got = _np(got)
    top = torch.finfo(DT[dtype]).max
    over = np.abs(want) > top
    bad = np.where(over, ~(np.isinf(got) | (np.abs(got) >= top)), np.abs(got - want) > bound)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])


# ------------------------------------------------------------------------------------ quantization
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,K", [(1, 16), (1, 128), (3, 144), (5, 2560), (333, 272), (2, 65536), (4097, 48)])
def test_quantize(T, K, dtype):
    import sparse_mixture_experts_gemv_gb300 as M
    x = _x(T, K, dtype)
    q, s = M.fp8_quantize(x)
    codes, scales = o.quantize(_np(x))
    np.testing.assert_array_equal(s.cpu().numpy(), scales)
    np.testing.assert_array_equal(_codes(q), codes)


def test_quantize_blocks_of_zeros_tiny_and_huge_values_ties_and_nan():
    import sparse_mixture_experts_gemv_gb300 as M
    x = torch.zeros(9, 256, device="cuda")
    x[1] = 1e-42            # the scale underflows to a denormal
    x[2, :128] = 1e-45      # and to 0: then it is 1
    x[3] = torch.linspace(-3e38, 3e38, 256, device="cuda")   # its step overflows: not finite in either block
    x[4, 0], x[4, 1:128] = 448, torch.from_numpy(((o._POSITIVE[1:] + o._POSITIVE[:-1]) / 2)).cuda().float().repeat(2)[:127]
    x[5, 3], x[6, 200], x[7, 130] = float("inf"), float("nan"), -float("inf")
    x[8] = -torch.linspace(0, 1e-40, 256, device="cuda")
    q, s = M.fp8_quantize(x)
    codes, scales = o.quantize(_np(x))
    np.testing.assert_array_equal(s.cpu().numpy(), scales)
    finite = np.isfinite(scales).repeat(128, 1)
    np.testing.assert_array_equal(_codes(q)[finite], codes[finite])
    assert s[5, 0].isnan() and s[6, 1].isnan() and s[7, 1].isnan()
    assert s[3].isnan().all() and int(s.isnan().sum()) == 5
    assert s[2, 0] == 1 and s[0, 0] == 1


def test_quantize_the_largest_values():
    import sparse_mixture_experts_gemv_gb300 as M
    x = torch.linspace(-3e38, 0, 256, device="cuda").repeat(2, 1)
    x[1] *= -1
    q, s = M.fp8_quantize(x)
    codes, scales = o.quantize(_np(x))
    assert np.isfinite(scales).all()
    np.testing.assert_array_equal(s.cpu().numpy(), scales)
    np.testing.assert_array_equal(_codes(q), codes)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,K", [(1, 512), (7, 80), (300, 400)])
def test_quantize_after_a_swiglu(T, K, dtype):
    import sparse_mixture_experts_gemv_gb300 as M
    x = (2 * torch.randn(T, 2 * K, generator=_gen(5), device="cuda")).to(DT[dtype])
    q, s = M.fp8_quantize(x, swiglu=True)
    h = o.swiglu(_np(x))
    codes, scales = o.quantize(h)
    # expf 2 ulp, the sum, the quotient and the product half each, twice over: below 8 * 2^-24 of the value
    np.testing.assert_allclose(s.cpu().numpy(), scales, rtol=10 * 2.0 ** -24)
    step = np.abs(_codes(q).astype(int) - codes.astype(int))
    assert step.max() <= 1 and (step > 0).mean() < 1e-3
    back = o.E4M3[_codes(q)] * _np(s).repeat(128, 1)[:, :K]
    np.testing.assert_allclose(back, h, rtol=2.0 ** -4 + 1e-5, atol=2.0 ** -10 * _np(s).max() * 1.01)


def test_quantize_rows_apart_and_none():
    import sparse_mixture_experts_gemv_gb300 as M
    x = _x(20, 400, "bf16")
    for v in (x[:, 8:264], x[:, 3:259], x[::3, :256], x.T[:256, :16], x[:1, :32].expand(20, 32)):
        q, s = M.fp8_quantize(v)
        codes, scales = o.quantize(_np(v))
        np.testing.assert_array_equal(_codes(q), codes)
        np.testing.assert_array_equal(s.cpu().numpy(), scales)
    q, s = M.fp8_quantize(x[:0])
    assert q.shape == (0, 400) and s.shape == (0, 4) and q.dtype is F8


# ---------------------------------------------------------------------------------------- products
SHAPES = [(1, 16, 1), (1, 128, 8), (1, 2048, 1024), (2, 144, 129), (17, 272, 77), (33, 128, 64), (65, 1040, 200),
          (127, 384, 256), (128, 256, 128), (129, 512, 257), (300, 2560, 1537), (1000, 128, 16), (40, 65536, 24),
          (1500, 400, 4104), (1300, 1024, 2056), (200, 512, 9000)]


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("T,K,N", SHAPES)
def test_matmul_of_quantized_rows(T, K, N, out):
    import sparse_mixture_experts_gemv_gb300 as M
    (x, xs), (w, ws) = _q(T, K), _w(N, K)
    got = M.fp8_matmul(x, w, ws, xs, DT[out])
    assert got.shape == (T, N) and got.dtype is DT[out]
    want, mag = o.matmul(_np(x), _np(xs), _np(w), _np(ws))
    _near(got, want, mag, K, out)
    assert torch.equal(got, M.fp8_matmul(x, w, ws, xs, DT[out]))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,K,N", [(1, 2048, 1024), (5, 144, 40), (130, 272, 300), (700, 512, 640)])
def test_matmul_quantizes_other_rows_as_fp8_quantize_does(T, K, N, dtype):
    import sparse_mixture_experts_gemv_gb300 as M
    x, (w, ws) = _x(T, K, dtype), _w(N, K)
    got = M.fp8_matmul(x, w, ws, out_dtype=torch.float32)
    codes, scales = o.quantize(_np(x))
    want, mag = o.matmul(o.E4M3[codes], scales, _np(w), _np(ws))
    _near(got, want, mag, K, "fp32")
    assert torch.equal(got, M.fp8_matmul(*[M.fp8_quantize(x)[0], w, ws, M.fp8_quantize(x)[1]], out_dtype=torch.float32))
    assert M.fp8_matmul(x, w, ws).dtype is DT[dtype]


def test_matmul_rows_apart():
    import sparse_mixture_experts_gemv_gb300 as M
    T, K, N = 50, 256, 96
    (x, xs), (w, ws) = _q(T, K), _w(N, K)
    want = M.fp8_matmul(x, w, ws, xs, torch.float32)

    def apart(t, pad, at):
        big = torch.zeros(t.shape[0], K + pad, dtype=torch.uint8, device="cuda")
        big[:, at:at + K] = t.view(torch.uint8)
        return big.view(F8)[:, at:at + K]
    for pad, at in ((16, 0), (32, 16), (5, 3), (16, 8)):
        assert torch.equal(M.fp8_matmul(apart(x, pad, at), apart(w, pad, at), ws, xs, torch.float32), want)
    turned = x.view(torch.uint8).T.contiguous().T.view(F8)
    assert torch.equal(M.fp8_matmul(turned, w, ws.T.contiguous().T, xs.T.contiguous().T, torch.float32), want)
    y = _x(T, K + 8, "bf16")
    assert torch.equal(M.fp8_matmul(y[:, 8:], w, ws), M.fp8_matmul(y[:, 8:].contiguous(), w, ws))
    assert torch.equal(M.fp8_matmul(y[:, 1:K + 1], w, ws), M.fp8_matmul(y[:, 1:K + 1].contiguous(), w, ws))


@pytest.mark.parametrize("T,N", [(3, 50), (200, 300)])
def test_nan_and_infinity_stay_in_their_rows_and_channels(T, N):
    import sparse_mixture_experts_gemv_gb300 as M
    (x, xs), (w, ws) = _q(T, 384), _w(N, 384)
    clean = M.fp8_matmul(x, w, ws, xs, torch.float32)
    x.view(torch.uint8)[1, 200] = 0x7F
    w.view(torch.uint8)[7, 3] = 0xFF
    got = M.fp8_matmul(x, w, ws, xs, torch.float32)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[1], bad[:, 7] = True, True
    assert bool(got[bad].isnan().all()) and torch.equal(got[~bad], clean[~bad])
    y = _x(T, 384, "bf16")
    clean = M.fp8_matmul(y, w, ws)
    y[2, 5] = float("inf")
    got = M.fp8_matmul(y, w, ws)
    assert bool(got[2].isnan().all())
    keep = [t for t in range(T) if t != 2]
    assert torch.equal(got[keep][:, :7], clean[keep][:, :7])


def test_scales_of_0_infinity_and_nan_are_arithmetic():
    import sparse_mixture_experts_gemv_gb300 as M
    (x, xs), (w, ws) = _q(6, 256), _w(130, 256)
    xs[0], xs[1, 1], xs[2, 0] = 0, float("nan"), float("inf")
    got = M.fp8_matmul(x, w, ws, xs, torch.float32)
    assert not got[0].any() and bool(got[1].isnan().all()) and not bool(got[2].isfinite().any())
    assert bool(got[3:].isfinite().all())


def test_no_rows_and_no_channels():
    import sparse_mixture_experts_gemv_gb300 as M
    (x, xs), (w, ws) = _q(4, 64), _w(8, 64)
    assert M.fp8_matmul(x[:0], w, ws, xs[:0]).shape == (0, 8)
    assert M.fp8_matmul(x, w[:0], ws[:0], xs).shape == (4, 0)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    (g, gs) = _w(2, 8, 64)
    assert M.fp8_grouped_matmul(x[:0], off, g, gs, xs[:0]).shape == (0, 8)
    assert M.fp8_grouped_matmul(x, off, g[:, :0].contiguous(), gs[:, :0].contiguous(), xs).shape == (4, 0)


def _offsets(counts):
    return torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32, device="cuda")


# counts of rows by expert, K, N: empty experts at the ends and between, tiles that end anywhere, one expert, many
GROUPS = [([1], 16, 8), ([8, 0, 0, 3], 128, 64), ([0, 0, 5, 0], 144, 72), ([128, 129, 0, 1, 300, 127], 272, 200),
          ([1] * 40, 256, 136), ([0] * 100 + [7] + [0] * 155, 512, 24), ([2000, 3], 128, 520), ([3] * 1024, 32, 16),
          ([40, 60, 16, 33, 64, 65], 640, 1000), ([0, 700, 0, 0, 900], 400, 128),
          ([(37 * i) % 301 for i in range(120)], 272, 200), ([17, 0, 33] * 30, 1168, 130),
          ([(53 * i) % 280 for i in range(120)], 512, 200)]


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("counts,K,N", GROUPS)
def test_grouped_matmul(counts, K, N, out):
    import sparse_mixture_experts_gemv_gb300 as M
    E, rows = len(counts), sum(counts)
    (x, xs), (w, ws) = _q(rows, K), _w(E, N, K)
    off = _offsets(counts)
    got = M.fp8_grouped_matmul(x, off, w, ws, xs, DT[out])
    want, mag = o.grouped_matmul(_np(x), _np(xs), off.tolist(), _np(w), _np(ws))
    _near(got, want, mag, K, out)
    # each expert's rows are those of a dense product with its weights
    e = int(np.argmax(counts))
    at = slice(int(off[e]), int(off[e + 1]))
    dense = M.fp8_matmul(x[at].contiguous(), w[e], ws[e], xs[at], DT[out])
    assert torch.equal(got[at], dense)


@pytest.mark.parametrize("dtype", list(DT))
def test_grouped_matmul_quantizes_other_rows(dtype):
    import sparse_mixture_experts_gemv_gb300 as M
    x, (w, ws), off = _x(200, 272, dtype), _w(5, 64, 272), _offsets([50, 0, 100, 1, 49])
    got = M.fp8_grouped_matmul(x, off, w, ws)
    q, s = M.fp8_quantize(x)
    assert got.dtype is DT[dtype] and torch.equal(got, M.fp8_grouped_matmul(q, off, w, ws, s, DT[dtype]))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,K,N", [(1, 16, 1), (1, 4096, 130), (2, 272, 77), (9, 144, 64), (15, 1040, 2000), (16, 1280, 260),
                                   (5, 4096, 96), (16, 1296, 40), (1, 4112, 24), (17, 128, 96), (3, 512, 20000)])
def test_few_rows_are_quantized_inside_the_product_to_the_same_bits(T, K, N, dtype):
    import sparse_mixture_experts_gemv_gb300 as M
    x, (w, ws) = _x(T, K + 8, dtype)[:, 8:], _w(N, K)
    q, s = M.fp8_quantize(x)
    for out in DT.values():
        assert torch.equal(M.fp8_matmul(x, w, ws, out_dtype=out), M.fp8_matmul(q, w, ws, s, out))
    want, mag = o.matmul(_np(q), _np(s), _np(w), _np(ws))
    _near(M.fp8_matmul(x, w, ws, out_dtype=torch.float32), want, mag, K, "fp32")


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("off", [[0, 3, 3, 8, 16], [2, 2, 5, 11, 12], [0, 16, 16, 16, 16], [0, 0, 0, 0, 1], [0, 0, 0, 0, 0], [7, 9, 3, 40, 12]])
@pytest.mark.parametrize("K,N", [(272, 77), (512, 200)])
def test_few_grouped_rows_likewise(off, K, N, dtype):
    import sparse_mixture_experts_gemv_gb300 as M
    x, (w, ws) = _x(16, K, dtype), _w(4, N, K)
    x[1, 3] = float("inf")   # stays in its row, and out of the result where the row has no expert
    q, s = M.fp8_quantize(x)
    off = torch.tensor(off, dtype=torch.int32, device="cuda")
    for out in DT.values():
        a, b = M.fp8_grouped_matmul(x, off, w, ws, out_dtype=out), M.fp8_grouped_matmul(q, off, w, ws, s, out)
        assert torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(0), b.nan_to_num(0))


@pytest.mark.parametrize("N", [64, 77])
def test_rows_of_no_expert_are_zeros(N):
    import sparse_mixture_experts_gemv_gb300 as M
    (x, xs), (w, ws) = _q(500, 128), _w(3, N, 128)
    off = torch.tensor([20, 120, 120, 333], dtype=torch.int32, device="cuda")
    x.view(torch.uint8)[:20] = 0x7F
    x.view(torch.uint8)[333:] = 0x7F
    for out in DT.values():
        torch.full((500, N), 7.0, dtype=out, device="cuda")   # what the output's memory may have held
        got = M.fp8_grouped_matmul(x, off, w, ws, xs, out)
        assert not got[:20].any() and not got[333:].any()
        assert torch.equal(got[20:120], M.fp8_matmul(x[20:120].contiguous(), w[0], ws[0], xs[20:120], out))
        assert torch.equal(got[120:333], M.fp8_matmul(x[120:333].contiguous(), w[2], ws[2], xs[120:333], out))
    none = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert not M.fp8_grouped_matmul(x, none, w, ws, xs).any()


def test_wrong_offsets_are_held_to_the_rows():
    """Below 0, past the rows, falling: what is outside is left out, what falls is an empty expert."""
    import sparse_mixture_experts_gemv_gb300 as M
    (x, xs), (w, ws) = _q(100, 128), _w(4, 32, 128)
    for wrong, right in (([-5, 50, 40, 60, 2 ** 31 - 1], [0, 50, 50, 60, 100]),
                         ([-2 ** 31, -1, 30, 10, 20], [0, 0, 30, 30, 30]), ([200, 0, 0, 0, 0], [100] * 5)):
        a = M.fp8_grouped_matmul(x, torch.tensor(wrong, dtype=torch.int32, device="cuda"), w, ws, xs)
        b = M.fp8_grouped_matmul(x, torch.tensor(right, dtype=torch.int32, device="cuda"), w, ws, xs)
        assert torch.equal(a, b)


def test_on_another_stream_captured_and_two_at_once():
    import sparse_mixture_experts_gemv_gb300 as M
    x, (w, ws), off = _x(300, 512, "bf16"), _w(4, 256, 512), _offsets([100, 0, 150, 50])
    want = M.fp8_grouped_matmul(x, off, w, ws)
    dense = M.fp8_matmul(x, w[0], ws[0])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        a = M.fp8_grouped_matmul(x, off, w, ws, stream=streams[0])
        b = M.fp8_matmul(x, w[0], ws[0], stream=streams[1])
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(b, dense)
    graphs, held = [], []
    for s in streams:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            held.append((M.fp8_grouped_matmul(x, off, w, ws), M.fp8_matmul(x, w[0], ws[0]), *M.fp8_quantize(x, True)))
    x.copy_(_x(300, 512, "bf16", 77))
    off.copy_(_offsets([0, 300, 0, 0]))
    for s, g in zip(streams, graphs):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    want = (M.fp8_grouped_matmul(x, off, w, ws), M.fp8_matmul(x, w[0], ws[0]), *M.fp8_quantize(x, True))
    for h in held:
        for a, b in zip(h, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert M.fp8_sync_status() == M.MOE_OK


def test_refusals():
    import sparse_mixture_experts_gemv_gb300 as M
    (x, xs), (w, ws), off = _q(4, 128), _w(3, 40, 128), _offsets([1, 2, 1])
    y = _x(4, 128, "bf16")
    for call in (lambda: M.fp8_quantize(y.double()), lambda: M.fp8_quantize(y[0]), lambda: M.fp8_quantize(x),
                 lambda: M.fp8_quantize(y[:, :17], True), lambda: M.fp8_quantize(y[:, :0]),
                 lambda: M.fp8_matmul(x, w[0], ws[0]), lambda: M.fp8_matmul(y, w[0], ws[0], xs),
                 lambda: M.fp8_matmul(y, w, ws), lambda: M.fp8_matmul(y, w[0].float(), ws[0]),
                 lambda: M.fp8_matmul(y, w[0], ws[0].double()), lambda: M.fp8_matmul(y, w[0], ws[1:]),
                 lambda: M.fp8_matmul(y[:, :64], w[0], ws[0]), lambda: M.fp8_matmul(x, w[0], ws[0], xs[:3]),
                 lambda: M.fp8_matmul(x, w[0], ws[0], xs.double()), lambda: M.fp8_matmul(y, w[0], ws[0], None, torch.float64),
                 lambda: M.fp8_matmul(y, w[0].cpu(), ws[0]), lambda: M.fp8_matmul(y, w[0], ws[0].cpu()),
                 lambda: M.fp8_matmul(y[:, :72], w[0][:, :72], ws[0]), lambda: M.fp8_matmul(y.view(torch.float16).view(torch.int16), w[0], ws[0]),
                 lambda: M.fp8_grouped_matmul(y, off[:3], w, ws), lambda: M.fp8_grouped_matmul(y, off.long(), w, ws),
                 lambda: M.fp8_grouped_matmul(y, off.cpu(), w, ws), lambda: M.fp8_grouped_matmul(y, off, w[0], ws[0]),
                 lambda: M.fp8_grouped_matmul(y, off, w.view(torch.uint8).transpose(0, 1).contiguous().transpose(0, 1).view(F8), ws),
                 lambda: M.fp8_grouped_matmul(y, off[:1], w[:0], ws[:0])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(M.MoeError):
        M.fp8_quantize(y[:, :24].contiguous().repeat(1, 3)[:, :24].contiguous())


def test_a_wait_that_runs_out_is_reported_once_and_the_next_call_is_right():
    import sparse_mixture_experts_gemv_gb300 as M
    from sparse_mixture_experts_gemv_gb300 import _native as N
    (x, xs), (w, ws) = _q(3, 256), _w(40, 256)
    want = M.fp8_matmul(x, w, ws, xs)
    assert M.fp8_sync_status() == M.MOE_OK
    N.load().moe_block_test_force_wait_timeout(1)
    try:
        M.fp8_matmul(x, w, ws, xs)
    finally:
        N.load().moe_block_test_force_wait_timeout(0)
    assert M.fp8_sync_status() == M.MOE_ERR_TIMEOUT
    assert M.fp8_sync_status() == M.MOE_OK
    assert torch.equal(M.fp8_matmul(x, w, ws, xs), want)
