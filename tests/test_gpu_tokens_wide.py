"""combine_tokens and its gradients on rows of nearly 2^31 values."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def _memory_goes_back():
    """Tens of gigabytes, which the allocator would keep from what allocates without it."""
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype,H", [(torch.bfloat16, 2 ** 31 - 8), (torch.float32, 2 ** 31 - 4)])
def test_combine_and_its_gradients(dtype, H):
    """Whole numbers of few bits: results are exact, the dot product too (its terms are 0 but for a thousand of them)."""
    import sparse_mixture_experts_gemv_gb300 as M
    g = torch.Generator("cuda").manual_seed(1)
    y = torch.randint(-4, 5, (2, H), generator=g, device="cuda", dtype=torch.int8).to(dtype)
    pos = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[2.0, -3.0]], device="cuda")
    out = M.combine_tokens(y, pos, w)
    want = torch.zeros(H, dtype=dtype, device="cuda").add_(y[1], alpha=2).add_(y[0], alpha=-3)
    assert torch.equal(out[0], want)
    del out
    assert torch.equal(M.dispatch_tokens_backward(y, pos)[0], want.copy_(y[0]).add_(y[1]))
    d = want.zero_()[None]
    at = torch.cat([torch.arange(500, device="cuda"), torch.arange(H - 500, H, device="cuda")])
    d[0, at] = torch.randint(-4, 5, (1000,), generator=g, device="cuda").to(dtype)
    d_y, d_w = M.combine_tokens_backward(d, y, pos, w)
    assert torch.equal(d_w, (y[[1, 0]][:, at].float() @ d[0, at].float())[None])
    for row, f in ((1, 2.0), (0, -3.0)):
        assert torch.equal(d_y[row, at], f * d[0, at])
        assert int(d_y[row].count_nonzero()) == int(d[0].count_nonzero())
