"""Cases, plain forms and exact values of the operators that stand beside the
matrix product: the gated linear layer with its backward pass, the
orthogonalised update and the 4-bit matrix-vector product.

``own`` false: the operators' plain forms in elementary torch operations and
32 bits, rounded once at the end.  ``own`` true: the calls that a user makes
of this package.
"""
import math

import torch

own = False

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}

# Muon's odd polynomial a x + b x^3 + c x^5, five times
NS_COEFFICIENTS = (3.4445, -4.7750, 2.0315)
NS_STEPS = 5
NS_EPS = 1e-7


def listed():
    return [
        # one token through a layer's gate and up projections: decoding, where
        # reading both weights is all there is to do
        {"name": "gated_token", "op": "gated", "T": 1, "D": 4096, "F": 8192, "type": "bf16", "act": "silu"},
        # a few dozen sequences decoding together, a feed-forward width that no tile divides
        {"name": "gated_decode_batch", "op": "gated", "T": 48, "D": 2048, "F": 6000, "type": "fp16", "act": "silu"},
        # a prompt of 4096 tokens
        {"name": "gated_prompt", "op": "gated", "T": 4096, "D": 4096, "F": 8192, "type": "fp16", "act": "gelu_tanh"},
        # a training step of a small model on packed sequences: nothing is a multiple of a tile
        {"name": "gated_step_ragged", "op": "gated_step", "T": 1000, "D": 1032, "F": 2730, "type": "fp16", "act": "gelu_tanh"},
        # a training step of one large layer: the largest case
        {"name": "gated_step_large", "op": "gated_step", "T": 8192, "D": 4096, "F": 8192, "type": "bf16", "act": "silu"},
        # the optimiser's update of a small weight, from a 32-bit momentum
        {"name": "ns_small", "op": "ns", "batch": 1, "rows": 256, "cols": 256, "type": "fp32"},
        # the same of eight attention projections of one shape, taller than wide
        {"name": "ns_tall_batch", "op": "ns", "batch": 8, "rows": 2048, "cols": 1000, "type": "fp16"},
        # one square weight of a large layer
        {"name": "ns_square", "op": "ns", "batch": 1, "rows": 4096, "cols": 4096, "type": "bf16"},
        # one token through a 4-bit layer, symmetric weights
        {"name": "w4_token", "op": "w4", "M": 1, "N": 8192, "K": 4096, "group": 128, "zeros": False, "type": "fp16"},
        # sixteen sequences decoding together through a wide layer, weights with zero points
        {"name": "w4_decode_batch", "op": "w4", "M": 16, "N": 8192, "K": 8192, "group": 64, "zeros": True, "type": "bf16"},
        # a speculated handful of tokens, odd sizes, the smallest groups
        {"name": "w4_ragged", "op": "w4", "M": 5, "N": 5000, "K": 6016, "group": 32, "zeros": True, "type": "fp16"},
        # a prompt of 256 tokens through a 4-bit layer
        {"name": "w4_prompt", "op": "w4", "M": 256, "N": 4096, "K": 4096, "group": 128, "zeros": False, "type": "bf16"},
    ]


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 5e12, w["flops"] / 1e15)


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["gated", "gated_step", "ns", "w4"])
        if op in ("gated", "gated_step"):
            # widths are multiples of 8, except now and then
            step = rng.choice([8, 8, 64, 1])
            case = {"op": op, "T": spread(1, 8192), "D": step * spread(max(1, 64 // step), 8192 // step),
                    "F": step * spread(max(1, 64 // step), 16384 // step),
                    "type": rng.choice(["fp16", "bf16"]), "act": rng.choice(["silu", "gelu_tanh"])}
        elif op == "ns":
            case = {"op": op, "batch": spread(1, 8), "rows": spread(32, 4096), "cols": spread(32, 8192),
                    "type": rng.choice(["fp16", "bf16", "fp32"])}
        else:
            group = rng.choice([32, 64, 128])
            case = {"op": op, "M": spread(1, 512), "N": spread(64, 16384), "K": group * spread(2, 16384 // group),
                    "group": group, "zeros": rng.random() < 0.5, "type": rng.choice(["fp16", "bf16"])}
        if _cost(case) <= most:
            return case


def work(case):
    if case["op"] in ("gated", "gated_step"):
        T, D, F = case["T"], case["D"], case["F"]
        if case["op"] == "gated":
            return {"bytes": 2 * (T * D + 2 * F * D + T * F), "flops": 4 * T * D * F}
        # x, dh, both weights in; h, dx and both weights' gradients out; two
        # products forward, four backward
        return {"bytes": 2 * (2 * T * D + 4 * F * D + 2 * T * F), "flops": 12 * T * D * F}
    if case["op"] == "ns":
        # X X^T and the polynomial of it are symmetric: half of each is enough
        m, n = sorted((case["rows"], case["cols"]))
        size = 4 if case["type"] == "fp32" else 2
        return {"bytes": case["batch"] * m * n * (size + 2), "flops": case["batch"] * NS_STEPS * (3 * m * m * n + m ** 3)}
    M, N, K, g = case["M"], case["N"], case["K"], case["group"]
    scales = N * (K // g) * 2 * (2 if case["zeros"] else 1)
    return {"bytes": N * K // 2 + scales + 2 * M * (K + N), "flops": 2 * M * N * K}


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    t = TYPES[case["type"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device=dev).mul_(std)

    if case["op"] in ("gated", "gated_step"):
        T, D, F = case["T"], case["D"], case["F"]
        s = {"case": case, "x": normal(T, D).to(t), "w_gate": normal(F, D, std=D ** -0.5).to(t),
             "w_up": normal(F, D, std=D ** -0.5).to(t)}
        if case["op"] == "gated_step":
            s["dh"] = normal(T, F, std=0.1).to(t)
        return s
    if case["op"] == "ns":
        # a momentum: noise with a few directions that stand out of it
        b, r, c = case["batch"], case["rows"], case["cols"]
        k = min(8, r, c)
        g = normal(b, r, c) + torch.bmm(normal(b, r, k), normal(b, k, c)) * (1.0 / math.sqrt(max(r, c)))
        g = (g * 1e-3).to(t)
        return {"case": case, "g": g[0] if b == 1 else g}
    M, N, K, group = case["M"], case["N"], case["K"], case["group"]
    s = {"case": case, "x": normal(M, K).to(t),
         "q": torch.randint(0, 256, (N, K // 2), generator=gen, device=dev, dtype=torch.uint8),
         "scales": (torch.rand(N, K // group, generator=gen, device=dev) + 0.5).mul_(0.2 * K ** -0.5).to(t), "zeros": None}
    if case["zeros"]:
        s["zeros"] = torch.randint(4, 12, (N, K // group), generator=gen, device=dev).to(t)
    return s


def _activation(g, act):
    """act(g) and its derivative, of 32-bit values."""
    if act == "silu":
        z, dz = g, torch.ones_like(g)
    else:  # 0.5 g (1 + tanh(y)) = g / (1 + exp(-2 y)), y = sqrt(2 / pi) (g + 0.044715 g^3)
        c = 2.0 * math.sqrt(2.0 / math.pi)
        z, dz = c * (g + 0.044715 * g * g * g), c * (1.0 + 3 * 0.044715 * g * g)
    s = 1.0 / (1.0 + torch.exp(-z))
    return g * s, s + g * s * (1.0 - s) * dz


def _plain(state):
    case = state["case"]
    t = TYPES[case["type"]]
    if case["op"] in ("gated", "gated_step"):
        x, wg, wu = (state[k].float() for k in ("x", "w_gate", "w_up"))
        g, u = x @ wg.t(), x @ wu.t()
        a, da = _activation(g, case["act"])
        h = (a * u).to(t)
        if case["op"] == "gated":
            return h
        dh = state["dh"].float()
        dg, du = dh * u * da, dh * a
        return {"h": h, "dx": (dg @ wg + du @ wu).to(t), "dw_gate": (dg.t() @ x).to(t), "dw_up": (du.t() @ x).to(t)}
    if case["op"] == "ns":
        a, b, c = NS_COEFFICIENTS
        g = state["g"].float()
        tall = g.shape[-2] > g.shape[-1]
        x = g.mT.contiguous() if tall else g
        norm = x.double().square().sum(dim=(-2, -1), keepdim=True).sqrt()
        x = (x.double() / (norm + NS_EPS)).float()
        for _ in range(NS_STEPS):
            p = x @ x.mT.contiguous()
            x = a * x + (b * p + c * (p @ p)) @ x
        return (x.mT if tall else x).to(torch.bfloat16).contiguous()
    q, group = state["q"], case["group"]
    w = torch.stack((q & 15, q >> 4), dim=-1).reshape(case["N"], -1, group).float()
    zero = 8.0 if state["zeros"] is None else state["zeros"].float()[:, :, None]
    w = (w - zero) * state["scales"].float()[:, :, None]
    return (state["x"].float() @ w.reshape(case["N"], case["K"]).t()).to(t)


def run(state):
    if not own:
        return _plain(state)
    import dense_fp16_gemm_04_amd as fw
    case = state["case"]
    if case["op"] == "gated":
        return fw.gated_nt(state["x"], state["w_gate"], state["w_up"], activation=case["act"])
    if case["op"] == "gated_step":
        h, saved = fw.gated_nt_train(state["x"], state["w_gate"], state["w_up"], activation=case["act"])
        dx, dw_gate, dw_up = fw.gated_nt_backward(state["dh"], state["x"], state["w_gate"], state["w_up"], saved)
        return {"h": h, "dx": dx, "dw_gate": dw_gate, "dw_up": dw_up}
    if case["op"] == "ns":
        return fw.orthogonalize_ns(state["g"], steps=NS_STEPS, coefficients=NS_COEFFICIENTS, eps=NS_EPS)
    return fw.gemv_w4(state["x"], state["q"], state["scales"], state["zeros"])


def exact(case, seed):
    """The definitions in 64 bits: gradients by automatic differentiation,
    the polynomial in nested form, the 4-bit product group by group."""
    s = prepare(case, seed)
    if case["op"] in ("gated", "gated_step"):
        leaves = [s[k].double().requires_grad_(case["op"] == "gated_step") for k in ("x", "w_gate", "w_up")]
        x, wg, wu = leaves
        g = torch.matmul(x, wg.transpose(0, 1))
        if case["act"] == "silu":
            a = g * torch.sigmoid(g)
        else:
            a = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g.pow(3))))
        h = a * torch.matmul(x, wu.transpose(0, 1))
        if case["op"] == "gated":
            return h
        dx, dwg, dwu = torch.autograd.grad(h, leaves, s["dh"].double())
        return {"h": h.detach(), "dx": dx, "dw_gate": dwg, "dw_up": dwu}
    if case["op"] == "ns":
        a, b, c = NS_COEFFICIENTS
        y = s["g"].double()
        y = y / (torch.linalg.matrix_norm(y, keepdim=True) + NS_EPS)
        if y.shape[-1] > y.shape[-2]:
            y = y.transpose(-2, -1).contiguous()
        for _ in range(NS_STEPS):  # y [long, short]: y <- y (a + s (b + c s)), s = y^T y
            gram = torch.matmul(y.transpose(-2, -1).contiguous(), y)
            inner = c * gram
            inner.diagonal(dim1=-2, dim2=-1).add_(b)
            poly = torch.matmul(gram, inner)
            poly.diagonal(dim1=-2, dim2=-1).add_(a)
            y = torch.matmul(y, poly)
        return (y.transpose(-2, -1) if s["g"].shape[-1] > s["g"].shape[-2] else y).contiguous()
    M, N, K, group = case["M"], case["N"], case["K"], case["group"]
    codes = torch.empty(N, K, dtype=torch.float64, device=s["q"].device)
    codes[:, 0::2] = (s["q"] % 16).double()
    codes[:, 1::2] = torch.div(s["q"], 16, rounding_mode="floor").double()
    x = s["x"].double()
    y = torch.zeros(M, N, dtype=torch.float64, device=x.device)
    for k in range(K // group):
        part = x[:, k * group:(k + 1) * group]
        dot = part @ codes[:, k * group:(k + 1) * group].t()
        zero = s["zeros"][:, k].double() if case["zeros"] else torch.full((N,), 8.0, dtype=torch.float64, device=x.device)
        y += s["scales"][:, k].double() * (dot - part.sum(dim=1, keepdim=True) * zero)
    return y
