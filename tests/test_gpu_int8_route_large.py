"""Offsets past 32 bits: the last rows of tensors with more than 2^31 elements."""
import numpy as np
import pytest

from oracle import route_int8_oracle as o

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def _np(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("T", [1, 6, 40])
def test_weights_past_32_bits(T):
    import sparse_mixture_experts_gemv_gb300 as M
    n, K = 1_060_000, 2048                       # 2.17e9 bytes
    w = torch.zeros(n, K, dtype=torch.int8, device="cuda")
    g = torch.Generator().manual_seed(T)
    w[-300:] = torch.randint(-127, 128, (300, K), generator=g, dtype=torch.int8).cuda()
    ws = torch.ones(n, device="cuda")
    x = torch.randint(-20, 21, (T, K), generator=g, dtype=torch.int8).cuda()
    xs = torch.full((T,), 0.5, device="cuda")
    got = M.int8_matmul(x, w, ws, xs, out_dtype=torch.float32)
    ref = o.matmul(_np(x), _np(w[-300:]), np.ones(300), _np(xs))
    assert (_np(got[:, -300:]) == ref).all()     # whole numbers and halves below 2^24: exact
    assert (got[:, :-300] == 0).all()
    del w, got
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T", [2, 30])
def test_experts_past_32_bits(T):
    import sparse_mixture_experts_gemv_gb300 as M
    E, H, I = 1024, 2048, 528                    # gate_up 2.2e9 bytes
    g = torch.Generator().manual_seed(T)

    def ints(*shape):
        return torch.randint(-127, 128, shape, generator=g, dtype=torch.int8).cuda()

    gate_up = torch.zeros(E, 2 * I, H, dtype=torch.int8, device="cuda")
    down = torch.zeros(E, H, I, dtype=torch.int8, device="cuda")
    gate_up[-2:], down[-2:] = ints(2, 2 * I, H), ints(2, H, I)
    gus, ds = torch.full((E, 2 * I), 3e-5, device="cuda"), torch.full((E, H), 1e-3, device="cuda")
    x = torch.randn(T, H, generator=g).bfloat16().cuda()
    idx = torch.tensor([[E - 1, E - 2]] * T, dtype=torch.int32, device="cuda")
    w = torch.full((T, 2), 0.5, device="cuda")
    got = M.int8_experts(x, idx, w, gate_up, gus, down, ds)
    small = idx - (E - 2)
    want = M.int8_experts(x, small, w, gate_up[-2:].clone(), gus[-2:].clone(), down[-2:].clone(), ds[-2:].clone())
    assert torch.equal(got, want) and got.abs().max() > 0
    del gate_up, down
    torch.cuda.empty_cache()


def test_logits_past_32_bits():
    import sparse_mixture_experts_gemv_gb300 as M
    T, E, k = 4_300_000, 512, 4                  # 2.2e9 logits
    x = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    x[-50:] = torch.randn(50, E, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    idx, w = M.route_experts(x, k)
    ref, rw = o.route(x[-50:].float().cpu().numpy(), k)
    assert (idx[-50:].cpu().numpy() == ref).all() and np.allclose(w[-50:].cpu().numpy(), rw, rtol=2.0 ** -16)
    d = torch.zeros(T, k, device="cuda")
    d[-50:] = torch.randn(50, k, generator=torch.Generator().manual_seed(1)).cuda()
    dx = M.route_experts_backward(d, x, idx)
    want = M.route_experts_backward(d[-50:].clone(), x[-50:].clone(), idx[-50:].clone())
    assert torch.equal(dx[-50:], want) and (dx[:-50] == 0).all()
    del x, dx, idx, w, d
    torch.cuda.empty_cache()
