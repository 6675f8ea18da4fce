"""The oracle of the routing rules and the 8-bit operators on worked examples, and the
operators' refusals, which come before anything touches a device."""
import ctypes

import numpy as np
import pytest

from oracle import route_int8_oracle as o

INF = float("inf")


def test_oracle_choice_worked_examples():
    assert o.choose([1.0, 3.0, 3.0, 2.0], 3, "softmax") == [1, 2, 3]          # equal ones by index
    assert o.choose([1.0, -INF, float("nan"), 2.0], 4, "sigmoid") == [3, 0, 1, 2]
    assert o.choose([0.0, 0.0, 0.0, 0.0], 2, "sigmoid", bias=[0, 0.1, 0, 0.2]) == [3, 1]
    # two groups: the second has the larger sum of two, the first the largest single
    x = [5.0, -9.0, 2.0, 2.0]
    assert o.choose(x, 2, "sigmoid", groups=2, top_groups=1, group_top=2) == [2, 3]
    assert o.choose(x, 2, "sigmoid", groups=2, top_groups=1, group_top=1) == [0, 1]
    # a group with one expert on has that one's key alone; one with none is last
    assert o.choose([-INF, -INF, -INF, 0.0], 2, "sigmoid", groups=2, top_groups=1) == [3, 2]


def test_oracle_weights_worked_examples():
    w = o.weights([0.0, np.log(3.0), -INF], [1, 0], "softmax")
    assert np.allclose(w, [0.75, 0.25])
    assert np.allclose(o.weights([0.0, 0.0, -INF], [0, 2], "sigmoid", scale=2.0), [2.0, 0.0])
    assert np.allclose(o.weights([0.0, 0.0], [0], "sigmoid", renormalise=False), [0.5])
    assert np.allclose(o.weights([-INF, -INF], [0, 1], "softmax"), 0)
    assert np.allclose(o.weights([INF, 0.0], [0, 1], "softmax"), [1, 0])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_oracle_gradient_against_differences(score, renormalise):
    rng = np.random.default_rng(3)
    x, d = rng.normal(size=(3, 9)), rng.normal(size=(3, 4))
    idx, _ = o.route(x, 4, score)
    got, _ = o.route_backward(d, x, idx, score, renormalise, 1.5)
    step = 1e-6
    for t in range(3):
        for e in range(9):
            hi, lo = x[t].copy(), x[t].copy()
            hi[e] += step
            lo[e] -= step
            diff = (o.weights(hi, idx[t], score, renormalise, 1.5) - o.weights(lo, idx[t], score, renormalise, 1.5))
            assert abs(got[t, e] - (diff * d[t]).sum() / (2 * step)) < 1e-8


def test_oracle_quantize_worked_examples():
    q, s, _ = o.quantize([[127.0, 0.5, 1.5, -2.5, -127.0], [0, 0, 0, 0, 0]])
    assert s.tolist() == [1.0, 1.0]
    assert q.tolist() == [[127, 0, 2, -2, -127], [0, 0, 0, 0, 0]]
    assert np.allclose(o.matmul(np.array([[2, 3]]), np.array([[1, -1], [4, 5]]), [0.5, 2.0], [10.0]), [[-5, 460]])


def _route_cfg(N, E=256, k=8, score=0, groups=1, top_groups=1, group_top=2, renormalise=1, scale=1.0):
    return ctypes.byref(N.moe_route_config_t(E, k, score, groups, top_groups, group_top, renormalise, scale))


def test_route_refusals():
    from sparse_mixture_experts_gemv_gb300 import _native as N
    f, fake = N.load().moe_route_experts, 0x10000   # never dereferenced
    inv, uns = N.MOE_ERR_INVALID_ARG, N.MOE_ERR_UNSUPPORTED

    def call(cfg, logits=fake, dtype=0, stride=256, bias=None, T=4, idx=fake, w=fake):
        return f(cfg, logits, dtype, stride, bias, T, idx, w, None)

    assert call(None) == inv
    for kw in ({"k": 0}, {"E": 0}, {"groups": 0}, {"groups": 3}, {"top_groups": 2}, {"group_top": 3}, {"score": 2},
               {"groups": 8, "top_groups": 1, "k": 33}, {"E": 4}, {"scale": INF}, {"scale": float("nan")}):
        assert call(_route_cfg(N, **kw)) == inv, kw
    for kw in ({"E": 513}, {"k": 33}, {"groups": 64, "top_groups": 8}):
        assert call(_route_cfg(N, **kw), stride=1024) == uns, kw
    ok = _route_cfg(N)
    assert call(ok, T=-1) == inv
    assert call(ok, logits=None) == inv and call(ok, logits=fake + 2) == inv and call(ok, dtype=3) == inv
    assert call(ok, stride=255) == inv
    assert call(ok, idx=None) == inv and call(ok, w=None) == inv and call(ok, w=fake + 2) == inv
    assert call(ok, bias=fake + 1) == inv
    assert call(ok, T=0, logits=None, idx=None, w=None) == N.MOE_OK
    b = N.load().moe_route_experts_backward
    assert b(ok, fake, 0, 256, None, fake, 4, fake, None) == inv
    assert b(ok, fake, 0, 256, fake, None, 4, fake, None) == inv
    assert b(ok, fake, 1, 256, fake, fake, 4, fake + 1, None) == inv
    assert b(ok, None, 0, 256, None, None, 0, None, None) == N.MOE_OK


def test_quant_matmul_refusals():
    from sparse_mixture_experts_gemv_gb300 import _native as N
    inv, uns = N.MOE_ERR_INVALID_ARG, N.MOE_ERR_UNSUPPORTED
    fake, far = 0x100000, 0x4000000
    need = ctypes.c_int64(-1)
    ws = N.load().moe_quant_matmul_workspace
    assert ws(4, 8, 64, 1, None) == inv and ws(-1, 8, 64, 1, ctypes.byref(need)) == inv
    assert ws(4, 8, 64, 4, ctypes.byref(need)) == inv
    assert ws(4000, 8, 64, 1, ctypes.byref(need)) == N.MOE_OK and need.value >= 0

    def call(x=fake, xd=1, xst=64, xs=None, w=2 * fake, wst=64, wsc=3 * fake, out=far, od=1, T=4, n=8, K=64, wsp=None,
             wsb=0):
        return N.load().moe_quant_matmul(x, xd, xst, xs, w, wst, wsc, out, od, T, n, K, wsp, wsb, None)

    for kw in ({"x": None}, {"w": None}, {"wsc": None}, {"out": None}, {"x": fake + 2}, {"w": fake + 8},
               {"out": far + 1}, {"wsc": fake + 1}, {"xd": 4}, {"od": 3}, {"xst": 63}, {"xst": 65}, {"wst": 48},
               {"wst": 72}, {"T": -1}, {"n": -1}, {"K": 0}, {"xs": fake}, {"xd": 3}, {"out": fake}, {"out": 2 * fake}):
        assert call(**kw) == inv, kw
    assert call(K=72, xst=80, wst=80) == uns
    assert call(K=65536 + 16, xst=65552, wst=65552) == uns
    assert call(T=0) == N.MOE_OK and call(n=0) == N.MOE_OK
    big = dict(T=4096, n=4096, K=2048, xst=2048, wst=2048, x=1 << 30, w=2 << 30, out=3 << 30)
    assert ws(4096, 4096, 2048, 1, ctypes.byref(need)) == N.MOE_OK
    if need.value:   # a workspace that is missing, too small or misaligned
        assert call(**big) == inv
        assert call(**big, wsp=4 << 30, wsb=need.value - 1) == inv
        assert call(**big, wsp=(4 << 30) + 16, wsb=need.value) == inv


def test_quant_experts_refusals():
    from sparse_mixture_experts_gemv_gb300 import _native as N
    inv, uns = N.MOE_ERR_INVALID_ARG, N.MOE_ERR_UNSUPPORTED
    fake = 0x100000
    need = ctypes.c_int64()

    def call(E=4, k=2, H=64, I=32, x=fake, xd=1, idx=fake, wt=fake, out=8 * fake, T=3, ws=9 * fake, wsb=1 << 30,
             gu=fake, gus=fake, dn=fake, dns=fake):
        cfg, w = N.moe_int8_experts_config_t(E, k, H, I), N.moe_int8_experts_weights_t(gu, gus, dn, dns)
        return N.load().moe_quant_experts(ctypes.byref(cfg), ctypes.byref(w), x, xd, idx, wt, out, T, ws, wsb, None)

    for kw in ({"E": 0}, {"k": 0}, {"H": 0}, {"I": -16}, {"T": -1}, {"xd": 0}, {"xd": 3}, {"x": None}, {"idx": None},
               {"wt": None}, {"out": None}, {"gu": None}, {"gus": None}, {"dn": None}, {"dns": None}, {"ws": None},
               {"wsb": 0}, {"x": fake + 2}, {"out": 8 * fake + 8}, {"gu": fake + 4}, {"ws": 9 * fake + 128},
               {"out": fake}, {"idx": fake + 1}):
        assert call(**kw) == inv, kw
    for kw in ({"H": 72}, {"I": 40}, {"k": 33}, {"E": 1025}, {"H": 16400}, {"I": 16400}):
        assert call(**kw) == uns, kw
    assert call(T=0, x=None, ws=None) == N.MOE_OK
    ws = N.load().moe_quant_experts_workspace
    assert ws(None, 1, ctypes.byref(need)) == inv


def test_python_calls_refuse_host_tensors_and_wrong_types():
    import torch
    import sparse_mixture_experts_gemv_gb300 as M
    with pytest.raises(ValueError):
        M.route_experts(torch.zeros(2, 8), 2)
    with pytest.raises(ValueError):
        M.int8_matmul(torch.zeros(2, 16), torch.zeros(4, 16, dtype=torch.int8), torch.ones(4))
    with pytest.raises(ValueError):
        M.int8_experts(torch.zeros(2, 16), None, None, None, None, None, None)
