"""Sizes that the C entry points cannot take are refused by the Python calls before anything is allocated."""
import pytest

torch = pytest.importorskip("torch")

F8, I32 = torch.float8_e4m3fn, torch.int32
FAR = 2 ** 32 + 5   # as a 32-bit integer it is 5


class Sized:
    """A CUDA tensor without gaps as far as the calls look at it: shape, type and place, no memory."""

    is_cuda, requires_grad, device = True, False, torch.device("cuda", 0)

    def __init__(self, shape, dtype=torch.float32):
        self.shape, self.dtype = torch.Size(shape), dtype

    def get_device(self):
        return 0

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def stride(self):
        return tuple(self.shape[i + 1:].numel() for i in range(len(self.shape)))

    def data_ptr(self):
        return 1 << 40

    def is_contiguous(self):
        return True

    def contiguous(self):
        return self


def _dispatch(M, T, k, H=1, n=None):
    return M.dispatch_tokens(Sized((T, H), torch.uint8), Sized((T, k), I32), 4, None if n is None else Sized((T, n)))


def _combine(M, T, k, H):
    return M.combine_tokens(Sized((T * k, H), torch.float16), Sized((T, k), I32), Sized((T, k)))


def _combine_backward(M, T, k, H):
    return M.combine_tokens_backward(Sized((T, H), torch.float16), Sized((T * k, H), torch.float16), Sized((T, k), I32),
                                     Sized((T, k)))


def _matmul(M, T, K, N, dtype=F8):
    return M.fp8_matmul(Sized((T, K), dtype), Sized((N, K), F8), Sized((-(-N // 128), -(-K // 128))),
                        Sized((T, -(-K // 128))) if dtype is F8 else None)


def _grouped(M, rows, E, K, N):
    return M.fp8_grouped_matmul(Sized((rows, K), F8), Sized((E + 1,), I32), Sized((E, N, K), F8),
                                Sized((E, -(-N // 128), -(-K // 128))), Sized((rows, -(-K // 128))))


CALLS = [lambda M: _dispatch(M, FAR, 1), lambda M: _dispatch(M, 1, FAR), lambda M: _dispatch(M, 1, 1, 1, FAR),
         lambda M: _combine(M, FAR, 1, 1), lambda M: _combine(M, 1, FAR, 1), lambda M: _combine(M, 1, 1, FAR),
         lambda M: _combine_backward(M, FAR, 1, 1), lambda M: _combine_backward(M, 1, FAR, 1),
         lambda M: _combine_backward(M, 1, 1, FAR),
         lambda M: M.dispatch_tokens_backward(Sized((FAR, 1)), Sized((FAR, 1), I32)),
         lambda M: M.dispatch_tokens_backward(Sized((1, FAR)), Sized((1, 1), I32)),
         lambda M: M.fp8_quantize(Sized((FAR, 16))), lambda M: M.fp8_quantize(Sized((1, 2 ** 32 + 16))),
         lambda M: M.fp8_quantize(Sized((1, 2 * (2 ** 32 + 16))), True),
         lambda M: _matmul(M, FAR, 16, 1), lambda M: _matmul(M, 1, 2 ** 32 + 16, 1), lambda M: _matmul(M, 1, 16, FAR),
         lambda M: _matmul(M, FAR, 16, 1, torch.bfloat16),
         lambda M: _grouped(M, FAR, 2, 16, 1), lambda M: _grouped(M, 2, FAR, 16, 1), lambda M: _grouped(M, 2, 2, 2 ** 32 + 16, 1),
         lambda M: _grouped(M, 2, 2, 16, FAR)]


@pytest.mark.parametrize("call", CALLS)
def test_sizes_past_32_bits_are_refused(call, monkeypatch):
    import sparse_mixture_experts_gemv_gb300 as M
    from sparse_mixture_experts_gemv_gb300 import _tensors
    monkeypatch.setattr(_tensors, "_device", lambda: 0)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: pytest.fail("allocated first"))
    with pytest.raises(ValueError, match="2\\^31"):
        call(M)


def test_numbers_of_choices_that_are_not_supported_are_refused_before_the_rows_are_allocated(monkeypatch):
    import sparse_mixture_experts_gemv_gb300 as M
    from sparse_mixture_experts_gemv_gb300 import _tensors
    monkeypatch.setattr(_tensors, "_device", lambda: 0)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: pytest.fail("allocated first"))
    for T, k in ((2 ** 30, 1), (3, 33)):
        with pytest.raises(M.MoeError):
            _dispatch(M, T, k)


def _int8_matmul(M, T, K, N):
    return M.int8_matmul(Sized((T, K), torch.int8), Sized((N, K), torch.int8), Sized((N,)), Sized((T,)))


def _int8_experts(M, T, k, E, H, I):
    return M.int8_experts(Sized((T, H), torch.bfloat16), Sized((T, k), I32), Sized((T, k)), Sized((E, 2 * I, H), torch.int8),
                          Sized((E, 2 * I)), Sized((E, H, I), torch.int8), Sized((E, H)))


EARLIER = [lambda M: _int8_matmul(M, FAR, 16, 1), lambda M: _int8_matmul(M, 1, 2 ** 32 + 16, 1), lambda M: _int8_matmul(M, 1, 16, FAR),
           lambda M: _int8_experts(M, FAR, 1, 2, 16, 16), lambda M: _int8_experts(M, 1, FAR, 2, 16, 16),
           lambda M: _int8_experts(M, 1, 1, FAR, 16, 16), lambda M: _int8_experts(M, 1, 1, 2, 2 ** 32 + 16, 16),
           lambda M: _int8_experts(M, 1, 1, 2, 16, 2 ** 32 + 16),
           lambda M: M.route_experts(Sized((FAR, 2)), 1), lambda M: M.route_experts(Sized((1, FAR)), 1),
           lambda M: M.route_experts_backward(Sized((FAR, 1)), Sized((FAR, 2)), Sized((FAR, 1), I32)),
           lambda M: M.route_experts_backward(Sized((1, 1)), Sized((1, FAR)), Sized((1, 1), I32))]


@pytest.mark.parametrize("call", EARLIER)
def test_sizes_past_32_bits_are_refused_by_the_other_tensor_calls(call, monkeypatch):
    test_sizes_past_32_bits_are_refused(call, monkeypatch)


def test_dispatch_refuses_rows_and_scales_past_a_gigabyte():
    """In the library, before anything reaches a device: a row's bytes, and its scales' likewise."""
    from sparse_mixture_experts_gemv_gb300 import _native as N
    far = [0x10000 + (i << 40) for i in range(8)]   # never read

    def dispatch(row, scales):
        return N.load().moe_dispatch_tokens(far[0], row, row, far[1] if scales else None, scales, far[2], 1, 1, 4, far[3],
                                            far[4] if scales else None, far[5], far[6], None, 0, None)
    assert [dispatch(2 ** 30, 0), dispatch(2 ** 31, 0), dispatch(16, 2 ** 28), dispatch(16, 2 ** 31 - 1)] == [N.MOE_ERR_UNSUPPORTED] * 4
