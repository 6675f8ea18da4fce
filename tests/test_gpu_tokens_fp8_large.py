"""Rows and results whose places pass 32 bits: more than 2^31 elements, and more than 2^32 bytes."""
import numpy as np
import pytest

from oracle import tokens_fp8_oracle as o

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def test_dispatch_and_combine():
    """560,000 rows of 4,096: 2.29e9 elements. Rows are looked at by samples and, all of them, by a sum that is exact."""
    import sparse_mixture_experts_gemv_gb300 as M
    T, k, E, H = 70000, 8, 64, 4096
    x = torch.randint(-8, 9, (T, H), generator=_gen(1), device="cuda", dtype=torch.int8).to(torch.bfloat16)
    idx = torch.randint(-1, E, (T, k), generator=_gen(2), device="cuda", dtype=torch.int32)
    rows, offsets, pos = M.dispatch_tokens(x, idx, E)
    on = idx >= 0
    counts = torch.bincount(idx[on].long(), minlength=E)
    assert torch.equal(offsets[1:].long(), counts.cumsum(0)) and int(offsets[0]) == 0
    place = torch.where(on, pos, ~pos).flatten().long()
    assert torch.equal(place.sort().values, torch.arange(T * k, device="cuda"))
    for j in range(k):
        t = on[:, j].nonzero()[:, 0][-2000:]
        assert torch.equal(rows[pos[t, j].long()], x[t])
    assert not rows[int(offsets[-1]):].any()
    sums = rows.float().sum(0)                       # whole numbers: x's columns times the choices of their tokens
    want = (x.double() * on.sum(1, keepdim=True)).sum(0)
    assert (sums.double() - want).abs().max() <= T * k * 8 * 2.0 ** -24 * T * k   # one rounding an addition at worst
    w = torch.ones(T, k, device="cuda")
    out = M.combine_tokens(rows, pos, w)
    assert torch.equal(out, (x.float() * on.sum(1, keepdim=True)).to(torch.bfloat16))
    d_y, d_w = M.combine_tokens_backward(x, rows, pos, w)
    assert torch.equal(d_y, rows)
    norms = x.float().square().sum(1)                # whole numbers below 2^24: exact in any order
    assert torch.equal(d_w, norms[:, None] * on)


def test_quantize():
    """140,000 rows of 16,384: 2.29e9 values, the last ones among them."""
    import sparse_mixture_experts_gemv_gb300 as M
    T, K = 140000, 16384
    x = torch.empty(T, K, dtype=torch.bfloat16, device="cuda").normal_(generator=_gen(3))
    q, s = M.fp8_quantize(x)
    for at in (slice(0, 3), slice(65535, 65538), slice(T - 3, T)):
        codes, scales = o.quantize(x[at].double().cpu().numpy())
        np.testing.assert_array_equal(q[at].view(torch.uint8).cpu().numpy(), codes)
        np.testing.assert_array_equal(s[at].cpu().numpy(), scales)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_products(out):
    """600,000 rows of 4,000 results, dense and of two experts: the same rows in different places have the same bits."""
    import sparse_mixture_experts_gemv_gb300 as M
    T, K, N = 600000, 128, 4000
    part = (torch.randn(1000, K, generator=_gen(4), device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    x = part.view(torch.uint8).repeat(T // 1000, 1).view(torch.float8_e4m3fn)
    xs = torch.rand(1000, 1, generator=_gen(5), device="cuda").repeat(T // 1000, 1)
    w = (torch.randn(2, N, K, generator=_gen(6), device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    ws = torch.rand(2, 32, 1, generator=_gen(7), device="cuda")
    first = M.fp8_matmul(x[:1000].contiguous(), w[0], ws[0], xs[:1000], out)
    y = M.fp8_matmul(x, w[0], ws[0], xs, out)
    assert bool((y.view(-1, 1000, N) == first).all())
    cut = 400000
    y = M.fp8_grouped_matmul(x, torch.tensor([0, cut, T - 1000], dtype=torch.int32, device="cuda"), w, ws, xs, out)
    second = M.fp8_matmul(x[:1000].contiguous(), w[1], ws[1], xs[:1000], out)
    assert bool((y[:cut].view(-1, 1000, N) == first).all()) and bool((y[cut:T - 1000].view(-1, 1000, N) == second).all())
    assert not y[T - 1000:].any()
