"""Cases of the routing and 8-bit operators, their plain forms and their values in 64 bits.

`route_experts` (with `route_experts_backward`), `int8_matmul` and `int8_experts` of
sparse_mixture_experts_gemv_gb300 are timed and compared with the plain forms below: elementary
torch operations in 32 bits (the selection keys of the router in 64, since two experts' scores
can lie closer than 32 bits tell apart). `own` says which of the two `run` makes.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "int8": torch.int8}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "int8": 1}


# ------------------------------------------------------------------------------------------ cases

def _route(name, T, E, k, score, dtype, bias=False, groups=1, top_groups=1, group_top=2, renormalise=True, scale=1.0,
           grad=False):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "score": score, "dtype": dtype, "bias": bias,
            "groups": groups, "top_groups": top_groups, "group_top": group_top, "renormalise": renormalise,
            "scale": scale, "grad": grad}


def _matmul(name, T, K, N, dtype, out):
    return {"name": name, "op": "matmul", "T": T, "K": K, "N": N, "dtype": dtype, "out": out}


def _experts(name, T, E, k, H, I, dtype):
    return {"name": name, "op": "experts", "T": T, "E": E, "k": k, "H": H, "I": I, "dtype": dtype}


def listed():
    return [
        # one decoded token of the Qwen-shaped layer: latency alone
        _route("route_decode", 1, 256, 8, "softmax", "fp32"),
        # a verification window of the Ling-shaped layer under a balance bias and expert groups
        _route("route_window_groups", 4, 512, 8, "sigmoid", "fp32", True, 8, 4, 2, True, 2.5),
        # one prefill chunk of the Qwen-shaped layer
        _route("route_prefill", 4096, 256, 8, "softmax", "fp32"),
        # a long batch of bf16 logits, where equal logits are common
        _route("route_long_bf16", 65536, 512, 8, "sigmoid", "bf16", True, 8, 4, 2, True, 2.5),
        # a training step's routing, forward and backward, over an odd number of tokens
        _route("route_train", 8191, 256, 8, "sigmoid", "fp32", True, 8, 4, 2, True, 1.0, True),
        # one token through a shared expert's gate and up rows
        _matmul("matmul_token", 1, 2048, 1024, "bf16", "bf16"),
        # one token through the 157,184 x 2,560 output projection
        _matmul("matmul_lm_head", 1, 2560, 157184, "bf16", "fp32"),
        # an odd chunk and an odd number of channels
        _matmul("matmul_odd", 333, 2560, 1537, "fp16", "fp16"),
        # a prefill chunk whose tokens come quantized already
        _matmul("matmul_prefill", 4096, 2048, 4096, "int8", "bf16"),
        # one decoded token through the Qwen-shaped layer's experts
        _experts("experts_decode", 1, 256, 8, 2048, 512, "bf16"),
        # a verification window through the Ling-shaped layer's experts
        _experts("experts_window", 4, 512, 8, 2560, 768, "bf16"),
        # one prefill chunk through the Qwen-shaped layer's experts
        _experts("experts_prefill", 4096, 256, 8, 2048, 512, "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["route", "route", "matmul", "matmul", "experts"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        per = rng.choice([8, 15, 16, 20, 32, 48, 64]) if groups > 1 else rng.choice([16, 60, 64, 128, 160, 256, 384, 512])
        E = min(512, groups * per)
        E -= E % groups
        top = rng.randint(1, groups) if groups > 1 else 1
        k = rng.randint(1, min(8, E // groups * top))
        grad = rng.random() < 0.4
        # the one weight of k = 1, renormalised, is a constant: its gradient would be rounding alone
        c = _route("", _log(rng, 1, 32768 if grad else 65536), E, k, rng.choice(["softmax", "sigmoid"]),
                   rng.choice(["fp32", "bf16", "fp16"]), rng.random() < 0.6, groups, top, rng.choice([1, 2]),
                   k > 1 and rng.random() < 0.7, rng.choice([1.0, 2.5]), grad)
    elif op == "matmul":
        K, N = 16 * _log(rng, 8, 256), _log(rng, 128, 16384)
        T = _log(rng, 1, max(1, min(4096, 4096 * 2048 * 4096 // (K * N))))
        c = _matmul("", T, K, N, rng.choice(["bf16", "fp16", "fp32", "int8"]), rng.choice(["bf16", "fp16", "fp32"]))
    else:
        E = rng.choice([16, 60, 64, 128, 256])
        H, I = 128 * rng.randint(2, 16), 32 * rng.randint(3, 24)
        k = rng.randint(1, 8)
        T = _log(rng, 1, max(1, min(4096, 32768 * 2048 * 512 // (k * H * I))))
        c = _experts("", T, E, k, H, I, rng.choice(["bf16", "fp16"]))
    del c["name"]
    return c


# ----------------------------------------------------------------------------------------- inputs

def _activations(T, K, g):
    """Normed hidden states: N(0, 1) with one channel in 256 ten times as large."""
    x = torch.randn(T, K, generator=g, device="cuda")
    return x * (1 + 9 * (torch.rand(K, generator=g, device="cuda") < 1 / 256))


def _weight(rows, K, g):
    """Rows as they are after a quantization by each row's largest value (about four deviations), and their scales."""
    w = torch.empty(*rows, K, dtype=torch.float16, device="cuda").normal_(generator=g)
    w = w.mul_(32).clamp_(-127, 127).round_().to(torch.int8)
    return w, 0.02 / 32 * (0.8 + 0.4 * torch.rand(*rows, generator=g, device="cuda"))


def prepare(case, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    s = {"case": case}
    T = case["T"]
    if case["op"] == "route":
        E = case["E"]
        popular = 0.5 * torch.randn(E, generator=g, device="cuda")
        s["logits"] = (torch.randn(T, E, generator=g, device="cuda") + popular).to(DTYPES[case["dtype"]])
        # a balance bias works against the popular experts, in steps of 1/1000
        size = 0.1 if case["score"] == "sigmoid" else 0.1 / E
        s["bias"] = (-popular * size * 1000).round() / 1000 if case["bias"] else None
        if case["grad"]:
            s["d_weights"] = torch.randn(T, case["k"], generator=g, device="cuda")
    elif case["op"] == "matmul":
        x = _activations(T, case["K"], g)
        if case["dtype"] == "int8":
            s["x"], s["x_scale"] = _quantize(x)
            s["x"] = s["x"].to(torch.int8)
        else:
            s["x"], s["x_scale"] = x.to(DTYPES[case["dtype"]]), None
        s["w"], s["w_scale"] = _weight((case["N"],), case["K"], g)
    else:
        E, H, I = case["E"], case["H"], case["I"]
        s["x"] = _activations(T, H, g).to(DTYPES[case["dtype"]])
        s["gate_up"], s["gate_up_scale"] = _weight((E, 2 * I), H, g)
        s["down"], s["down_scale"] = _weight((E, H), I, g)
        # a balanced router's choices: each token's own, some experts a few times as popular as others
        score = torch.randn(T, E, generator=g, device="cuda") + 0.3 * torch.randn(E, generator=g, device="cuda")
        top, idx = score.topk(case["k"], dim=1)
        s["idx"], s["weights"] = idx.to(torch.int32), torch.softmax(top, dim=1)
    return s


# ------------------------------------------------------------------------------------ plain forms

def _quantize(x):
    """Whole numbers of -127..127 (held in 32-bit floats) and a scale for each row. The quotient is taken in
    64 bits: half of a row's largest value lies next to the border between two whole numbers."""
    amax = x.abs().amax(dim=-1)
    scale = torch.where(amax > 0, amax / 127, torch.ones_like(amax))
    return (x.double() / scale.unsqueeze(-1).double()).round().clamp(-127, 127).float(), scale


def _top(key, k):
    """The k largest of each row in descending order, equal ones by index."""
    return key.sort(dim=-1, descending=True, stable=True).indices[..., :k]


def _plain_route(logits, k, score, bias, groups, top_groups, group_top, renormalise, scale):
    x = logits.double()
    s = torch.softmax(x, dim=-1) if score == "softmax" else torch.sigmoid(x)
    if bias is None and groups == 1:
        idx = _top(x, k)
    else:
        key = s if bias is None else s + bias.double()
        if groups > 1:
            T, E = x.shape
            g = key.view(T, groups, E // groups)
            best = g.sort(dim=-1, descending=True).values[..., :group_top].sum(-1)
            kept = torch.zeros_like(best, dtype=torch.bool).scatter_(1, _top(best, top_groups), True)
            key = key.masked_fill(~kept.repeat_interleave(E // groups, dim=1), -math.inf)
        idx = _top(key, k)
    w = s.gather(1, idx)
    if renormalise:
        w = w / w.sum(-1, keepdim=True)
    return idx.to(torch.int32), (w * scale).float()


def _plain_route_backward(d_weights, logits, idx, score, renormalise, scale):
    x, at = logits.float(), idx.long()
    s = torch.softmax(x, dim=-1) if score == "softmax" else torch.sigmoid(x)
    d, chosen = d_weights * scale, s.gather(1, at)
    if renormalise:
        total = chosen.sum(-1, keepdim=True)
        d = (d - (d * chosen).sum(-1, keepdim=True) / total) / total
    ds = torch.zeros_like(s).scatter_(1, at, d)
    if score == "softmax":
        dx = s * (ds - (d * chosen).sum(-1, keepdim=True))
    else:
        dx = s * (1 - s) * ds
    return dx.to(logits.dtype)


def _plain_matmul(x, w, w_scale, x_scale, out_dtype):
    q, x_scale = _quantize(x.float()) if x_scale is None else (x.float(), x_scale)
    return (q @ w.float().T * x_scale[:, None] * w_scale).to(out_dtype)


def _plain_expert_rows(q, q_scale, gate_up, gate_up_scale, down, down_scale):
    """[B, n, H] quantized rows through the B experts' weights."""
    a = torch.bmm(q, gate_up.float().transpose(1, 2)) * q_scale[..., None] * gate_up_scale[:, None]
    gate, up = a.chunk(2, dim=-1)
    h, h_scale = _quantize(gate / (1 + torch.exp(-gate)) * up)
    return torch.bmm(h, down.float().transpose(1, 2)) * h_scale[..., None] * down_scale[:, None]


def _plain_experts(x, idx, weights, gate_up, gate_up_scale, down, down_scale):
    T, k = idx.shape
    E = gate_up.shape[0]
    q, q_scale = _quantize(x.float())
    flat = idx.reshape(-1).long()
    if T * k <= E // 4:  # few rows: each with its own expert's weights
        q, q_scale = q.repeat_interleave(k, 0)[:, None], q_scale.repeat_interleave(k, 0)[:, None]
        y = _plain_expert_rows(q, q_scale, gate_up[flat], gate_up_scale[flat], down[flat], down_scale[flat])[:, 0]
    else:  # rows grouped by expert, every group as long as the longest
        e, order = flat.sort(stable=True)
        counts = torch.bincount(flat, minlength=E)
        at = torch.arange(T * k, device=x.device) - (counts.cumsum(0) - counts)[e]
        longest = int(counts.max())
        rows = q.new_zeros(E, longest, q.shape[1])
        rows[e, at] = q[order // k]
        row_scale = q.new_ones(E, longest)
        row_scale[e, at] = q_scale[order // k]
        y = torch.empty(T * k, q.shape[1], device=x.device)
        y[order] = _plain_expert_rows(rows, row_scale, gate_up, gate_up_scale, down, down_scale)[e, at]
    return (y.view(T, k, -1) * weights[..., None]).sum(1).to(x.dtype)


# -------------------------------------------------------------------------------------------- run

def run(s):
    c = s["case"]
    if own:
        import sparse_mixture_experts_gemv_gb300 as M
    if c["op"] == "route":
        if own:
            idx, w = M.route_experts(s["logits"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                                     top_groups=c["top_groups"], group_top=c["group_top"],
                                     renormalise=c["renormalise"], scale=c["scale"])
        else:
            idx, w = _plain_route(s["logits"], c["k"], c["score"], s["bias"], c["groups"], c["top_groups"],
                                  c["group_top"], c["renormalise"], c["scale"])
        out = {"idx": idx, "weights": w}
        if c["grad"]:
            back = M.route_experts_backward if own else _plain_route_backward
            out["d_logits"] = back(s["d_weights"], s["logits"], idx, c["score"], c["renormalise"], c["scale"])
        return out
    if c["op"] == "matmul":
        product = M.int8_matmul if own else _plain_matmul
        return product(s["x"], s["w"], s["w_scale"], s["x_scale"], DTYPES[c["out"]])
    experts = M.int8_experts if own else _plain_experts
    return experts(s["x"], s["idx"], s["weights"], s["gate_up"], s["gate_up_scale"], s["down"], s["down_scale"])


def work(case):
    T = case["T"]
    if case["op"] == "route":
        row = case["E"] * BYTES[case["dtype"]]
        b = T * (row + 8 * case["k"]) + (4 * case["E"] if case["bias"] else 0)
        if case["grad"]:  # d_weights in, d_logits out
            b += T * (row + 4 * case["k"])
        return {"bytes": b, "flops": 4 * T * case["E"] * (2 if case["grad"] else 1)}
    if case["op"] == "matmul":
        K, N = case["K"], case["N"]
        return {"bytes": T * K * BYTES[case["dtype"]] + N * K + 4 * N + T * N * BYTES[case["out"]] +
                (4 * T if case["dtype"] == "int8" else 0), "flops": 2 * T * K * N}
    E, k, H, I = case["E"], case["k"], case["H"], case["I"]
    touched = E * (1 - (1 - k / E) ** T)  # experts that at least one token chose
    return {"bytes": touched * (3 * I * H + 8 * I + 4 * H) + 4 * T * H + 8 * T * k, "flops": 6 * T * k * H * I}


# -------------------------------------------------------------------------------- values in 64 bits

def _exact_scale(rows):
    """A row's scale is held in 32 bits: that is part of the definition."""
    top = rows.abs().max(dim=-1, keepdim=True).values
    top[top == 0] = 127.0
    return (top / 127).float().double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        # given the chosen experts, which are whole numbers and compared as such
        idx = _exact_choice(s).long()
        x = s["logits"].to(torch.float64)
        if case["score"] == "sigmoid":
            p = 1.0 / (1.0 + torch.exp(-x))
        else:
            p = torch.exp(x - torch.logsumexp(x, 1, keepdim=True))
        top = torch.stack([p[torch.arange(len(p), device=p.device), idx[:, j]] for j in range(case["k"])], 1)
        z = top.sum(1, keepdim=True) if case["renormalise"] else torch.ones_like(top[:, :1])
        out = {"idx": None, "weights": case["scale"] * top / z}
        if case["grad"]:
            # the Jacobian row by row of the chosen: dw_j/dp_i = scale (delta_ij / z - [renormalised] p_j / z^2)
            d = s["d_weights"].to(torch.float64) * case["scale"]
            dp = d / z
            if case["renormalise"]:
                dp = dp - (d * top).sum(1, keepdim=True) / z ** 2
            full = torch.zeros_like(p)
            full[torch.arange(len(p), device=p.device)[:, None], idx] = dp
            out["d_logits"] = full * p * (1 - p) if case["score"] == "sigmoid" else \
                p * full - p * (p * full).sum(1, keepdim=True)
        return out
    if case["op"] == "matmul":
        x, scale = s["x"].to(torch.float64), s["x_scale"]
        if scale is None:
            scale = _exact_scale(x)
            x = torch.round(x / scale)
        else:
            scale = scale.double()[:, None]
        out = torch.empty(case["T"], case["N"], dtype=torch.float64, device="cuda")
        for at in range(0, case["N"], 16384):
            w = s["w"][at:at + 16384].double() * s["w_scale"][at:at + 16384].double()[:, None]
            out[:, at:at + 16384] = (x * scale) @ w.T
        return out
    x = s["x"].to(torch.float64)
    scale = _exact_scale(x)
    x = torch.round(x / scale) * scale
    out = torch.zeros_like(x)
    for e in torch.unique(s["idx"]).tolist():
        t, j = (s["idx"] == e).nonzero(as_tuple=True)
        a = x[t] @ (s["gate_up"][e].double() * s["gate_up_scale"][e].double()[:, None]).T
        half = a.shape[1] // 2
        h = a[:, :half] * torch.sigmoid(a[:, :half]) * a[:, half:]
        scale = _exact_scale(h)
        h = torch.round(h / scale) * scale
        y = h @ (s["down"][e].double() * s["down_scale"][e].double()[:, None]).T
        out[t] += s["weights"][t, j].double()[:, None] * y  # a token chooses an expert once
    return out


def _exact_choice(s):
    """The experts that the definition chooses, found without a sort: k times the largest key that is left."""
    c, x = s["case"], s["logits"].double()
    T, E = x.shape
    if s["bias"] is None and c["groups"] == 1:
        key = x.clone()
    else:
        key = 1 / (1 + torch.exp(-x)) if c["score"] == "sigmoid" else torch.softmax(x, 1)
        if s["bias"] is not None:
            key = key + s["bias"].double()
    if c["groups"] > 1:
        left = key.view(T, c["groups"], -1).clone()
        best = torch.zeros(T, c["groups"], dtype=torch.float64, device=x.device)
        for _ in range(min(c["group_top"], left.shape[2])):
            v, at = left.max(dim=2)
            best += v
            left.scatter_(2, at[..., None], -math.inf)
        off = torch.ones_like(best, dtype=torch.bool)
        for _ in range(c["top_groups"]):
            first = (best == best.max(1, keepdim=True).values).int().argmax(1, keepdim=True)
            off.scatter_(1, first, False)
            best.scatter_(1, first, -math.inf)
        key = torch.where(off[..., None], -math.inf, key.view(T, c["groups"], -1)).view(T, E)
    chosen = []
    for _ in range(c["k"]):
        first = (key == key.max(1, keepdim=True).values).int().argmax(1, keepdim=True)
        chosen.append(first)
        key.scatter_(1, first, -math.inf)
    return torch.cat(chosen, 1)
