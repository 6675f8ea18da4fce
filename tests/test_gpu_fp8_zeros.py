"""Zeros below zero in the 8-bit floating-point quantization: -0 / scale is -0, and its E4M3 code 0x80, as elementary
operations on tensors have it and the oracle does."""
import numpy as np
import pytest

from oracle import tokens_fp8_oracle as o

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def _codes(t):
    return t.view(torch.uint8).cpu().numpy()


def _x(T, K, dtype):
    """Rows with both zeros in ordinary blocks, and a block of -0 alone."""
    x = torch.randn(T, K, generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    x[:, 1::5], x[:, 3::7] = -0.0, 0.0
    x[-1, :128] = -0.0
    return x.to(DT[dtype])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,K", [(1, 16), (3, 272), (500, 144)])
def test_quantize(T, K, dtype):
    import sparse_mixture_experts_gemv_gb300 as M
    x = _x(T, K, dtype)
    q, s = M.fp8_quantize(x)
    codes, scales = o.quantize(x.double().cpu().numpy())
    np.testing.assert_array_equal(s.cpu().numpy(), scales)
    np.testing.assert_array_equal(_codes(q), codes)
    plain = (x.float()[:, :128 * (K // 128)].view(T, -1, 128) / s[:, :K // 128, None]).to(torch.float8_e4m3fn)
    assert torch.equal(q[:, :128 * (K // 128)].view(torch.uint8), plain.view(T, -1).view(torch.uint8))


@pytest.mark.parametrize("dtype", list(DT))
def test_quantize_values_that_vanish_keep_their_signs(dtype):
    """Quotients that are 0 in E4M3, some of them in 32 bits."""
    import sparse_mixture_experts_gemv_gb300 as M
    x = torch.zeros(2, 128, device="cuda")
    x[:, 0] = 60000.0
    x[0, 1:64] = -torch.logspace(-7, 0, 63, device="cuda")
    x[1, 64:] = -0.0
    if dtype != "fp16":
        x[1, 1:40] = -torch.logspace(-44, -20, 39, device="cuda")
        x[1, 0] = 1e28
    x = x.to(DT[dtype])
    q, s = M.fp8_quantize(x)
    codes, scales = o.quantize(x.double().cpu().numpy())
    np.testing.assert_array_equal(s.cpu().numpy(), scales)
    np.testing.assert_array_equal(_codes(q), codes)


@pytest.mark.parametrize("dtype", list(DT))
def test_quantize_after_a_swiglu(dtype):
    """-0 from the gate, from the up half, from both (then it is 0), in blocks of either side of the gate's border of -80."""
    import sparse_mixture_experts_gemv_gb300 as M
    K = 128
    x = torch.randn(4, 2 * K, generator=torch.Generator("cuda").manual_seed(2), device="cuda").to(DT[dtype])
    g, u = x[:, :K], x[:, K:]
    g[:, 0:20], u[:, 10:30] = -0.0, -0.0
    g[:, 40:50], u[:, 45:60] = 0.0, 0.0
    u[:, 12], g[:, 25] = 2.0, 3.0
    g[2:, 100] = -90.0
    g[3] = -0.0
    q, s = M.fp8_quantize(x, swiglu=True)
    gf, uf = x.float().chunk(2, dim=1)
    h = gf / (1 + torch.exp(-gf)) * uf
    zero = (h == 0).cpu().numpy()
    assert zero.sum() > 100
    np.testing.assert_array_equal(_codes(q)[zero], np.where(np.signbit(h.cpu().numpy()), 0x80, 0)[zero])


def test_rows_quantized_inside_the_product_and_dispatched_are_unchanged():
    import sparse_mixture_experts_gemv_gb300 as M
    x = _x(5, 272, "bf16")
    w = (torch.randn(40, 272, device="cuda") * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    ws = torch.rand(1, 3, device="cuda")
    q, s = M.fp8_quantize(x)
    assert torch.equal(M.fp8_matmul(x, w, ws, out_dtype=torch.float32), M.fp8_matmul(q, w, ws, s, torch.float32))
    idx = torch.tensor([[0, 1]] * 5, dtype=torch.int32, device="cuda")
    rows, _, _, pos = M.dispatch_tokens(q, idx, 2, s)
    assert torch.equal(rows[pos[:, 1].long()].view(torch.uint8), q.view(torch.uint8))
