"""One sparse mixture-of-experts layer with experts in 8-bit floating point, put together from the package's
operators as a user would:

  idx, w = route_experts(x W_r, ...)                      the choices and their weights
  q, s   = fp8_quantize(x)                                E4M3, a scale for each block of 128
  rows, rs, offsets, pos = dispatch_tokens(q, idx, E, s)  tokens in the order of their experts
  a      = fp8_grouped_matmul(rows, offsets, gate_up, ..) the gate and up rows of each expert
  h, hs  = fp8_quantize(a, swiglu=True)                   silu(gate) * up, quantized again
  y      = fp8_grouped_matmul(h, offsets, down, ...)
  out    = combine_tokens(y, pos, w) + shared expert      (fp8_matmul twice)

and a training step of the router and of experts in bf16 through dispatch_tokens and combine_tokens, whose
gradients are the package's too. Run: python3 examples/fp8_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_mixture_experts_gemv_gb300 as moe  # noqa: E402

BLOCK = 128


def quantize_blocks(w):
    """Weights [..., N, K] -> E4M3 and a scale for each 128 x 128: a block's largest magnitude becomes 448."""
    n, k = w.shape[-2:]
    padded = torch.nn.functional.pad(w.float(), (0, -k % BLOCK, 0, -n % BLOCK))
    blocks = padded.unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, BLOCK))       # [..., N / 128, 128, K / 128, 128]
    scale = blocks.abs().amax((-3, -1)).clamp(min=1e-12) / 448
    q = (blocks / scale[..., :, None, :, None]).clamp(-448, 448).flatten(-4, -3).flatten(-2, -1)[..., :n, :k]
    return q.contiguous().to(torch.float8_e4m3fn), scale


def dequantize(q, scale):
    s = scale.repeat_interleave(BLOCK, -2)[..., :q.shape[-2], :].repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]
    return q.double() * s.double()


class Fp8Layer:
    """router [H, E], gate_up [E, 2I, H], down [E, H, I] and the shared expert's [2 Is, H] and [H, Is], any floating type."""

    def __init__(self, router, gate_up, down, shared_gate_up, shared_down, k):
        self.router, self.k, self.E = router.float(), k, gate_up.shape[0]
        self.gate_up, self.down = quantize_blocks(gate_up), quantize_blocks(down)
        self.shared_gate_up, self.shared_down = quantize_blocks(shared_gate_up), quantize_blocks(shared_down)

    def route(self, x):
        return moe.route_experts(x.float() @ self.router, self.k)

    def forward(self, x):
        idx, weights = self.route(x)
        q, scale = moe.fp8_quantize(x)
        rows, row_scale, offsets, pos = moe.dispatch_tokens(q, idx, self.E, scale)
        a = moe.fp8_grouped_matmul(rows, offsets, *self.gate_up, row_scale, torch.bfloat16)
        h, h_scale = moe.fp8_quantize(a, swiglu=True)
        y = moe.fp8_grouped_matmul(h, offsets, *self.down, h_scale, torch.bfloat16)
        out = moe.combine_tokens(y, pos, weights)
        a = moe.fp8_matmul(q, *self.shared_gate_up, scale, torch.bfloat16)
        h, h_scale = moe.fp8_quantize(a, swiglu=True)
        return out + moe.fp8_matmul(h, *self.shared_down, h_scale, out.dtype)


class TrainedLayer(torch.nn.Module):
    """Router and experts in bf16: dispatch and combine between them carry the gradients of both."""

    def __init__(self, H, E, I, k, device="cuda"):
        super().__init__()
        g = torch.Generator(device).manual_seed(7)

        def weight(*shape):
            return torch.nn.Parameter(shape[-1] ** -0.5 * torch.randn(*shape, generator=g, device=device))
        self.k, self.E = k, E
        self.router, self.gate_up, self.down = weight(E, H), weight(E, 2 * I, H), weight(E, H, I)

    def forward(self, x):
        idx, weights = moe.route_experts(x.float() @ self.router.T, self.k)
        rows, offsets, pos = moe.dispatch_tokens(x, idx, self.E)
        at = offsets.tolist()
        out = []
        for e in range(self.E):
            gate, up = (rows[at[e]:at[e + 1]] @ self.gate_up[e].to(x.dtype).T).chunk(2, dim=1)
            out.append((torch.nn.functional.silu(gate) * up) @ self.down[e].to(x.dtype).T)
        return moe.combine_tokens(torch.cat(out), pos, weights)


def make_layer(H=512, E=32, I=256, k=4, seed=0, device="cuda"):
    g = torch.Generator(device).manual_seed(seed)

    def rand(*shape):
        return 0.02 * torch.randn(*shape, generator=g, device=device)
    return Fp8Layer(rand(H, E) * 3, rand(E, 2 * I, H), rand(E, H, I), rand(2 * I, H), rand(H, I), k)


def plain_layer(layer, x, idx, w):
    """The layer with the weights that the 8 bits stand for, in 64 bits, one token at a time."""
    def expert(v, gate_up, down):
        gate, up = (gate_up @ v).chunk(2)
        return down @ (torch.nn.functional.silu(gate) * up)
    gate_up, down, sgu, sd = (dequantize(*q) for q in (layer.gate_up, layer.down, layer.shared_gate_up, layer.shared_down))
    return torch.stack([sum(w[t, j].double() * expert(v, gate_up[e], down[e]) for j, e in enumerate(idx[t].tolist())) +
                        expert(v, sgu, sd) for t, v in enumerate(x.double())])


def main():
    layer = make_layer()
    x = torch.randn(200, 512, generator=torch.Generator("cuda").manual_seed(1), device="cuda").bfloat16()
    idx, w = layer.route(x)
    want = plain_layer(layer, x, idx, w)
    worst = 0.0
    for tokens in (1, 4, 200):   # a decoded token, a verification window, a chunk of a prompt
        out = layer.forward(x[:tokens]).double()
        error = float((out - want[:tokens]).norm() / want[:tokens].norm())
        worst = max(worst, error)
        print(f"{tokens:4d} tokens: {error:.2%} from the layer without rounding of its activations")

    model = TrainedLayer(64, 8, 32, 2)
    tokens = torch.randn(100, 64, generator=torch.Generator("cuda").manual_seed(2), device="cuda")
    optimizer = torch.optim.SGD(model.parameters(), lr=0.1)
    for _ in range(3):
        optimizer.zero_grad()
        loss = (model(tokens) - tokens).square().mean()
        loss.backward()
        optimizer.step()
    norms = {n: float(p.grad.norm()) for n, p in model.named_parameters()}
    print("gradients of a training step:", ", ".join(f"{n} {v:.2e}" for n, v in norms.items()))
    assert moe.fp8_sync_status() == moe.MOE_OK
    return worst, norms


if __name__ == "__main__":
    main()
