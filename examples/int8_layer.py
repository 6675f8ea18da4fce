"""One sparse mixture-of-experts layer with another routing rule and with its experts in 8-bit
integers, put together from the package's operators as a user would:

  logits = x W_r                                   (the router's product, here torch's)
  idx, w = route_experts(logits, ...)              sigmoid scores, a bias for balance, expert groups
  out    = int8_experts(x, idx, w, ...)            the chosen experts, weights in int8
         + int8_matmul(...) twice                  an always-on shared expert

and one step of the router's training: the gradient of the logits through the weights, and the
bias moved against the experts' loads. Run: python3 examples/int8_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_mixture_experts_gemv_gb300 as moe  # noqa: E402


def quantize_channels(w):
    """Rows of weights -> int8 and a scale for each: the largest magnitude of a row becomes 127."""
    scale = w.float().abs().amax(-1) / 127
    return (w.float() / scale[..., None]).round().to(torch.int8), scale


class Int8Layer:
    """gate_up [E, 2I, H], down [E, H, I] and the shared expert's [2 Is, H] and [H, Is] in any floating type."""

    def __init__(self, router, gate_up, down, shared_gate_up, shared_down, k, groups, top_groups, scale):
        self.router = router.float()                       # [H, E]
        self.bias = torch.zeros(router.shape[1], device=router.device)
        self.gate_up, self.down = quantize_channels(gate_up), quantize_channels(down)
        self.shared_gate_up, self.shared_down = quantize_channels(shared_gate_up), quantize_channels(shared_down)
        self.rule = dict(score="sigmoid", groups=groups, top_groups=top_groups, renormalise=True, scale=scale)
        self.k = k

    def route(self, x):
        logits = x.float() @ self.router
        return logits, moe.route_experts(logits, self.k, bias=self.bias, **self.rule)

    def forward(self, x):
        _, (idx, weights) = self.route(x)
        out = moe.int8_experts(x, idx, weights.detach(), *self.gate_up, *self.down)
        gate, up = moe.int8_matmul(x, *self.shared_gate_up, out_dtype=torch.float32).chunk(2, dim=1)
        h = torch.nn.functional.silu(gate) * up
        return out + moe.int8_matmul(h, *self.shared_down, out_dtype=x.dtype)

    def router_gradient(self, x, d_weights):
        """d loss / d router from that of the routing weights, [T, k]."""
        logits, (idx, _) = self.route(x)
        d_logits = moe.route_experts_backward(d_weights, logits, idx, self.rule["score"], True, self.rule["scale"])
        return x.float().T @ d_logits

    def balance(self, idx, step=1e-3):
        """Moves the bias of every expert against its load: it chooses, and has no gradient."""
        load = torch.bincount(idx.flatten().long(), minlength=len(self.bias)).float()
        self.bias += step * torch.sign(load.mean() - load)


def make_layer(H=512, E=64, I=256, k=4, seed=0, device="cuda"):
    g = torch.Generator(device).manual_seed(seed)

    def rand(*shape):
        return 0.02 * torch.randn(*shape, generator=g, device=device)

    weights = rand(H, E) * 3, rand(E, 2 * I, H), rand(E, H, I), rand(2 * I, H), rand(H, I)
    return Int8Layer(*weights, k=k, groups=8, top_groups=4, scale=2.5), weights


def plain_layer(layer, weights, x, idx, w):
    """The same layer with the weights that the integers stand for, in 64 bits, one token at a time."""
    def real(q):
        return q[0].double() * q[1].double()[..., None]

    def expert(v, gate_up, down):
        gate, up = (gate_up @ v).chunk(2)
        return down @ (torch.nn.functional.silu(gate) * up)

    gate_up, down, sgu, sd = (real(q) for q in (layer.gate_up, layer.down, layer.shared_gate_up, layer.shared_down))
    return torch.stack([sum(w[t, j].double() * expert(v, gate_up[e], down[e]) for j, e in enumerate(idx[t].tolist())) +
                        expert(v, sgu, sd) for t, v in enumerate(x.double())])


def main():
    layer, weights = make_layer()
    x = torch.randn(300, 512, generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
    _, (idx, w) = layer.route(x)
    want = plain_layer(layer, weights, x, idx, w)
    worst = 0.0
    for tokens in (1, 4, 300):   # a decoded token, a verification window, a chunk of a prompt
        out = layer.forward(x[:tokens]).double()
        error = float((out - want[:tokens]).norm() / want[:tokens].norm())
        worst = max(worst, error)
        print(f"{tokens:4d} tokens: {error:.2%} from the layer without rounding of its activations")
    before = torch.bincount(idx.flatten().long(), minlength=64).float().std()
    for _ in range(30):
        layer.balance(layer.route(x)[1][0], step=0.01)
    after = torch.bincount(layer.route(x)[1][0].flatten().long(), minlength=64).float().std()
    grad = layer.router_gradient(x, torch.randn_like(w))
    print(f"loads deviate by {before:.1f}, balanced by {after:.1f}; |d router| {float(grad.norm()):.2e}")
    assert moe.int8_sync_status() == moe.MOE_OK
    return worst, float(before), float(after)


if __name__ == "__main__":
    main()
