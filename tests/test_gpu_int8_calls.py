"""int8_matmul and int8_experts: what they refuse, and the sizes at the ends of their ranges."""
import pytest

from test_gpu_int8 import DT, _choices, _experts, _ints, _scales, _x

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("T", [2, 40])
def test_inputs_that_record_a_gradient_are_refused(T):
    """Neither call has one: an output without a graph would train nothing, and say nothing."""
    import sparse_mixture_experts_gemv_gb300 as M
    x, w, ws = _x(T, 64, "bf16"), _ints(8, 64), _scales(8)
    q, qs = _ints(T, 64), _scales(T)
    (idx, weights), ex = _choices(T, 8, 2), _experts(8, 64, 32)
    xe = _x(T, 64, "bf16")

    def leaf(t):
        return t.clone().requires_grad_()

    calls = [lambda: M.int8_matmul(leaf(x), w, ws), lambda: M.int8_matmul(x, w, leaf(ws)),
             lambda: M.int8_matmul(q, w, ws, leaf(qs)), lambda: M.int8_experts(leaf(xe), idx, weights, *ex),
             lambda: M.int8_experts(xe, idx, leaf(weights), *ex),
             lambda: M.int8_experts(xe, idx, weights, ex[0], leaf(ex[1]), *ex[2:]),
             lambda: M.int8_experts(xe, idx, weights, *ex[:3], leaf(ex[3]))]
    for call in calls:
        with pytest.raises(ValueError, match="gradient"):
            call()
        with torch.no_grad():
            assert not call().requires_grad
    from torch.autograd import forward_ad
    with forward_ad.dual_level():
        with pytest.raises(ValueError, match="tangent"):
            M.int8_matmul(forward_ad.make_dual(x, torch.ones_like(x)), w, ws)
        with pytest.raises(ValueError, match="tangent"):
            M.int8_experts(xe, idx, forward_ad.make_dual(weights, torch.ones_like(weights)), *ex)


def test_tensors_freed_after_a_call_on_another_stream_are_not_handed_out_again():
    """Neither an input nor an output of a call on another stream is given to someone else while it is in use."""
    import sparse_mixture_experts_gemv_gb300 as M
    w, ws = _ints(64, 4096), _scales(64)
    s = torch.cuda.Stream()
    x = _x(64, 4096, "fp32")
    at, keep = x.data_ptr(), x.clone()
    M.int8_matmul(x, w, ws, stream=s)        # loads the kernels, which may wait for the GPU
    torch.full((64, 4096), 3.0, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(400_000_000)       # the call below waits behind this, some 0.2 s
    out = M.int8_matmul(x, w, ws, stream=s)
    del x
    again = [torch.full((64, 4096), 3.0, device="cuda") for _ in range(3)]
    assert not s.query()
    assert at not in [t.data_ptr() for t in again]
    s.synchronize()
    assert torch.equal(out, M.int8_matmul(keep, w, ws))


def test_most_rows_of_one_channel():
    """65,536 rows of a K that leaves a CTA one row: more than a grid's second dimension takes."""
    import sparse_mixture_experts_gemv_gb300 as M
    T, K = 65536, 49168
    g = torch.Generator("cuda").manual_seed(0)
    x = torch.randint(-127, 128, (T, K), generator=g, dtype=torch.int8, device="cuda")
    w, one, xs = _ints(1, K), torch.ones(1, device="cuda"), torch.full((T,), 0.5, device="cuda")
    got = M.int8_matmul(x, w, one, xs, out_dtype=torch.float32)
    some = torch.tensor([0, 1, 191, 192, 32767, 40000, 65534, 65535], device="cuda")
    ref = (x[some].double() * w.double()).sum(1) * 0.5
    assert (ref.abs() * 2 < 2 ** 24).all() and torch.equal(got[some, 0].double(), ref)   # exact below 2^24
    del x, got
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T", [1, 4])
def test_sums_of_few_tokens_are_exact(T):
    """Integer sums beyond 2^24, of one sign and cancelling: added as integers and rounded once."""
    import sparse_mixture_experts_gemv_gb300 as M
    K, n = 65536, 40
    w = torch.full((n, K), 127, dtype=torch.int8)
    w[1] = -128
    w[2, ::2] = -127
    w[3, : K // 2] = -127
    w[4:] = _ints(n - 4, K).cpu()
    x = torch.full((T, K), 127, dtype=torch.int8)
    x[T - 1, 1:] = -128
    got = M.int8_matmul(x.cuda(), w.cuda(), torch.ones(n, device="cuda"), torch.ones(T, device="cuda"),
                        out_dtype=torch.float32)
    ref = x.long() @ w.long().T
    assert ref.abs().max() > 2 ** 29 and torch.equal(got.cpu(), ref.float())


@pytest.mark.parametrize("T", [1, 40, 300])
def test_sums_that_no_part_of_passes_24_bits_are_exact(T):
    """K of 1,024 and less: the largest partial sum there can be is 128 * 128 * 1,024 = 2^24."""
    import sparse_mixture_experts_gemv_gb300 as M
    K, n = 1024, 2000
    w = _ints(n, K, lo=100).cpu()
    w[1], w[2], w[3, : K // 2] = -128, 127, -127
    w[4:600] = -_ints(596, K, lo=100, seed=1).cpu()
    x = _ints(T, K, lo=120, seed=2).cpu()
    x[0] = -128
    got = M.int8_matmul(x.cuda(), w.cuda(), torch.ones(n, device="cuda"), torch.ones(T, device="cuda"),
                        out_dtype=torch.float32)
    ref = (x.double() @ w.double().T).long()
    assert ref.abs().max() == 2 ** 24 and (T == 1 or (ref % 2 != 0).any())   # the row of -128 alone is even
    assert torch.equal(got.cpu().long(), ref)


@pytest.mark.parametrize("T", [2, 500])
@pytest.mark.parametrize("dtype", list(DT))
def test_rows_quantized_by_the_caller_are_the_calls(T, dtype):
    """amax / 127 on the GPU is the scale that the call takes, halves of the largest value among the elements."""
    import sparse_mixture_experts_gemv_gb300 as M
    x = _x(T, 272, dtype, seed=T)
    x[:, 7] = x.abs().amax(1) / 2
    w, ws = _ints(300, 272), _scales(300)
    scale = x.float().abs().amax(1) / 127
    q = (x.double() / scale.double()[:, None]).round().to(torch.int8)
    assert torch.equal(M.int8_matmul(x, w, ws, out_dtype=torch.float32),
                       M.int8_matmul(q, w, ws, scale, out_dtype=torch.float32))


@pytest.mark.parametrize("op", ["matmul", "experts"])
def test_a_wait_that_runs_out_is_reported_and_leaves_the_device_usable(op):
    """Tokens that never come: every role of the product winds down after its bounded wait, the status says so
    once, and the next call is right."""
    import sparse_mixture_experts_gemv_gb300 as M
    from sparse_mixture_experts_gemv_gb300 import _native as N
    if op == "matmul":
        x, w, ws = _x(200, 1040, "bf16"), _ints(3000, 1040), _scales(3000)
        call = lambda: M.int8_matmul(x, w, ws)  # noqa: E731
    else:
        xe, (idx, weights), ex = _x(40, 640, "bf16"), _choices(40, 8, 2), _experts(8, 640, 576)
        call = lambda: M.int8_experts(xe, idx, weights, *ex)  # noqa: E731
    want = call()
    assert M.int8_sync_status() == N.MOE_OK
    N.load().moe_quant_test_force_wait_timeout(1)
    try:
        call()
    finally:
        N.load().moe_quant_test_force_wait_timeout(0)
    assert M.int8_sync_status() == N.MOE_ERR_TIMEOUT
    assert M.int8_sync_status() == N.MOE_OK
    assert torch.equal(call(), want)
    assert M.int8_sync_status() == N.MOE_OK
