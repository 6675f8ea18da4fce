"""8-bit floating-point products whose rows or channels are counted near 2^31."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
F8 = torch.float8_e4m3fn
PERIOD = 128 * 1024   # channels or rows after which the inputs, and with them the results, repeat


@pytest.fixture(autouse=True)
def _memory_goes_back():
    """Tens of gigabytes, which the allocator would keep from what allocates without it."""
    yield
    torch.cuda.empty_cache()


def _part(rows, K, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(rows, K, generator=g, device="cuda") * 100).clamp(-448, 448).to(F8)


def _repeated(part, rows):
    """`rows` rows that repeat those of `part`."""
    out = torch.empty((rows, *part.shape[1:]), dtype=part.dtype, device="cuda")
    whole, bytes_ = rows // len(part), part.element_size() == 1
    a, p = (out.view(torch.uint8), part.view(torch.uint8)) if bytes_ else (out, part)
    a[:whole * len(p)].view(whole, *p.shape).copy_(p)
    a[whole * len(p):] = p[:rows - whole * len(p)]
    return out


@pytest.mark.parametrize("out,N", [(torch.float32, 2 ** 29 + 64), (torch.bfloat16, 2 ** 30 + 40), (torch.float16, 2 ** 30 + 9)])
@pytest.mark.parametrize("dtype", [F8, torch.bfloat16])
def test_channels_whose_bytes_pass_31_bits(dtype, out, N):
    """Three rows, whose results the warps store themselves: half a billion channels and more, every one compared. The
    memory of the results holds NaN before, so that a channel that is not written shows."""
    import sparse_mixture_experts_gemv_gb300 as M
    x, xs = _part(3, 16, 1), torch.rand(3, 1, generator=torch.Generator("cuda").manual_seed(2), device="cuda") + 0.1
    if dtype is not F8:
        x, xs = x.to(dtype), None
    part, scale = _part(PERIOD, 16, 3), torch.rand(PERIOD // 128, 1, generator=torch.Generator("cuda").manual_seed(4), device="cuda")
    first = M.fp8_matmul(x, part, scale, xs, out)
    w, ws = _repeated(part, N), _repeated(scale, -(-N // 128))
    torch.full((3, N), float("nan"), dtype=out, device="cuda")
    y = M.fp8_matmul(x, w, ws, xs, out)
    whole = N // PERIOD * PERIOD
    for t in range(3):
        assert bool((y[t, :whole].view(-1, PERIOD) == first[t]).all()) and torch.equal(y[t, whole:], first[t, :N - whole])


@pytest.mark.parametrize("dtype", [F8, torch.bfloat16])
def test_rows_counted_to_the_last(dtype):
    """2^31 - 1 rows of one channel, dense and of two experts with rows of none behind them."""
    import sparse_mixture_experts_gemv_gb300 as M
    T, cut, end = 2 ** 31 - 1, 9 * PERIOD, 2 ** 31 - 1 - PERIOD + 50
    part, scale = _part(PERIOD, 16, 1), torch.rand(PERIOD, 1, generator=torch.Generator("cuda").manual_seed(2), device="cuda") + 0.1
    w, ws = _part(2, 16, 3)[:, None].contiguous(), torch.rand(2, 1, 1, generator=torch.Generator("cuda").manual_seed(4), device="cuda")
    if dtype is not F8:
        part, scale = part.to(dtype), None
    first, second = (M.fp8_matmul(part, w[e], ws[e], scale, torch.bfloat16) for e in (0, 1))
    x, xs = _repeated(part, T), None if scale is None else _repeated(scale, T)
    whole = T // PERIOD * PERIOD
    y = M.fp8_matmul(x, w[0], ws[0], xs, torch.bfloat16)
    assert bool((y[:whole].view(-1, PERIOD, 1) == first).all()) and torch.equal(y[whole:], first[:T - whole])
    del y
    off = torch.tensor([0, cut, end], dtype=torch.int32, device="cuda")
    y = M.fp8_grouped_matmul(x, off, w, ws, xs, torch.bfloat16)
    assert bool((y[:cut].view(-1, PERIOD, 1) == first).all()) and not y[end:].any()
    whole = (end - cut) // PERIOD * PERIOD
    assert bool((y[cut:cut + whole].view(-1, PERIOD, 1) == second).all())
    assert torch.equal(y[cut + whole:end], second[:end - cut - whole])


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
def test_channels_counted_to_the_last(out):
    """2^31 - 2 channels, as many as a call takes; one more is refused."""
    import sparse_mixture_experts_gemv_gb300 as M
    test_channels_whose_bytes_pass_31_bits(F8, out, 2 ** 31 - 2)
    x, xs = _part(3, 16, 1), torch.rand(3, 1, device="cuda")
    w, ws = torch.empty(2 ** 31 - 1, 16, dtype=F8, device="cuda"), torch.empty(2 ** 24, 1, device="cuda")
    with pytest.raises(M.MoeError):
        M.fp8_matmul(x, w, ws, xs, out)
