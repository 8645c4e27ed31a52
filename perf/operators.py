"""Operators of a gated feed-forward block, as cases to be timed and compared.

Four operators, by the case's "op":

  gated       H = act(A G^T) * (A U^T)                       (16-bit weights, any number of tokens)
  gated_back  the gradients of sum(H * dH) by A, G and U     (the products of A are recomputed)
  w4          C = A W^T, W in 4 bits with group scales       (a few tokens)
  w4_gated    H = act(A G^T) * (A U^T), G and U as W         (a few tokens)

A is [M, K]; G, U and W are [N, K]; H, dH and C are [M, N].  Rows of the
16-bit matrices start on 16-byte boundaries, so an odd width is a slice of a
wider buffer.  W[n, k] = (q[n, k] - z[n, k // group]) * s[n, k // group] with
codes q in 0..15 (two per byte, even k in the low nibble), 16-bit scales s,
and zero points z in 0..15, or 8 throughout.
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one token through a narrow block: the launch and one pass over 16 MB of weights
        {"name": "gated_token", "op": "gated", "M": 1, "N": 4096, "K": 1024, "act": "silu", "dtype": "bf16"},
        # a decode batch of 16 requests: the weights are streamed once
        {"name": "gated_decode", "op": "gated", "M": 16, "N": 7168, "K": 4096, "act": "silu", "dtype": "bf16"},
        # a short prompt, every size odd
        {"name": "gated_ragged", "op": "gated", "M": 333, "N": 2741, "K": 1093, "act": "gelu", "dtype": "fp16"},
        # a long prompt, or a training batch's forward pass: bound by the tensor cores
        {"name": "gated_prompt", "op": "gated", "M": 8192, "N": 8192, "K": 4096, "act": "silu", "dtype": "bf16"},
        # a small block's training step: launches and few tiles
        {"name": "back_small", "op": "gated_back", "M": 128, "N": 1024, "K": 512, "act": "silu", "dtype": "bf16"},
        # a packed batch of ragged documents in fp16, every size odd
        {"name": "back_ragged", "op": "gated_back", "M": 1001, "N": 1397, "K": 2051, "act": "gelu", "dtype": "fp16"},
        # a training micro-batch: bound by the tensor cores
        {"name": "back_step", "op": "gated_back", "M": 4096, "N": 7168, "K": 4096, "act": "silu", "dtype": "bf16"},
        # one token through a square projection: latency
        {"name": "w4_token", "op": "w4", "M": 1, "N": 4096, "K": 4096, "group": 128, "zeros": False, "dtype": "bf16"},
        # a decode batch with the finest groups and zero points
        {"name": "w4_batch", "op": "w4", "M": 16, "N": 7168, "K": 4096, "group": 32, "zeros": True, "dtype": "fp16"},
        # one token through an output head of odd width: 270 MB of codes from memory
        {"name": "w4_head", "op": "w4", "M": 1, "N": 65537, "K": 8192, "group": 128, "zeros": False, "dtype": "bf16"},
        # one token through a quantised block's first half
        {"name": "w4_gated_token", "op": "w4_gated", "M": 1, "N": 7168, "K": 4096, "group": 128, "zeros": False,
         "act": "silu", "dtype": "bf16"},
        # five requests, zero points, a width that no tile divides
        {"name": "w4_gated_batch", "op": "w4_gated", "M": 5, "N": 5119, "K": 8320, "group": 64, "zeros": True,
         "act": "gelu", "dtype": "fp16"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated", "gated_back", "w4", "w4_gated"])
    case = {"op": op, "dtype": rng.choice(["bf16", "fp16"])}
    if op in ("gated", "gated_back"):
        # the listed largest: 8192 x 8192 x 4096 forward; a third of it for the
        # backward pass, which does three times the arithmetic
        most = 8192 * 8192 * 4096 // (1 if op == "gated" else 3)
        while True:
            M = _log_int(rng, 1, 8192)
            N = _log_int(rng, 200, 8192)
            K = _log_int(rng, 200, 8192)
            if M * N * K <= most:
                break
        if rng.random() < 0.5:  # a model's own widths are usually round
            N, K = (N + 63) // 64 * 64, (K + 63) // 64 * 64
            if M * N * K > most:
                M = max(1, most // (N * K))
        case.update(M=M, N=N, K=K, act=rng.choice(["silu", "gelu", "relu"]))
    else:
        M = _log_int(rng, 1, 32)
        K = 32 * _log_int(rng, 8, 512)
        N = _log_int(rng, 200, 65536 if op == "w4" else 16384)
        N = min(N, 65536 * 8192 // K)
        case.update(M=M, N=N, K=K, group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5)
        if op == "w4_gated":
            case["act"] = rng.choice(["silu", "gelu", "relu"])
    return case


def _rows(gen, rows, cols, dtype, scale):
    """[rows, cols], each row on a 16-byte boundary."""
    ld = (cols + 7) // 8 * 8
    t = torch.randn((rows, ld), generator=gen, device="cuda", dtype=torch.float32).mul_(scale)
    return t.to(dtype)[:, :cols]


def _activations(gen, rows, cols, dtype):
    """Normal values over channels of unequal size, a few of them several times the rest."""
    x = _rows(gen, rows, cols, torch.float32, 1.0)
    x = x * torch.exp(0.5 * torch.randn((1, cols), generator=gen, device="cuda"))
    ld = (cols + 7) // 8 * 8
    out = torch.zeros((rows, ld), device="cuda", dtype=dtype)
    out[:, :cols] = x.to(dtype)
    return out[:, :cols]


def _w4_weights(gen, case):
    N, K, group = case["N"], case["K"], case["group"]
    groups = (K + group - 1) // group
    codes = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.rand((N, groups), generator=gen, device="cuda").add_(0.5).mul_(0.25 / math.sqrt(K))
    zeros = None
    if case["zeros"]:
        zeros = torch.randint(4, 12, (N, groups), generator=gen, device="cuda", dtype=torch.uint8)
    return codes, scales.to(_TYPES[case["dtype"]]), zeros


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    dt = _TYPES[case["dtype"]]
    M, N, K = case["M"], case["N"], case["K"]
    s = {"case": case, "A": _activations(gen, M, K, dt)}
    if case["op"] in ("gated", "gated_back"):
        s["G"] = _rows(gen, N, K, dt, 1.0 / math.sqrt(K))
        s["U"] = _rows(gen, N, K, dt, 1.0 / math.sqrt(K))
        if case["op"] == "gated_back":
            s["dH"] = _rows(gen, M, N, dt, 1.0)
        return s
    names = ["W"] if case["op"] == "w4" else ["G", "U"]
    s["W4"] = [_w4_weights(gen, case) for _ in names]
    if own:
        # the weights as a serving program keeps them: packed once, at load
        import dense_gemm_preshuffle_gb300 as gp
        s["packed"] = [gp.preshuffle_w4g(codes, scales, case["group"], zeros=zeros) for codes, scales, zeros in s["W4"]]
        torch.cuda.synchronize()
    return s


# ------------------------------------------------------------ the plain forms

def _act(x, act):
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    return torch.where(x > 0, x, torch.zeros_like(x))


def _act_slope(x, act):
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-x))
        return s * (1.0 + x * (1.0 - s))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) * (1.0 / math.sqrt(2 * math.pi))
    return (x > 0).to(x.dtype)


def _dequantize(codes, scales, zeros, group, K):
    q = torch.stack((codes & 15, codes >> 4), dim=2).reshape(codes.shape[0], K).float()
    of = torch.arange(K, device=codes.device) // group
    z = 8.0 if zeros is None else zeros.float()[:, of]
    return (q - z) * scales.float()[:, of]


def _plain(s):
    case = s["case"]
    dt = _TYPES[case["dtype"]]
    A = s["A"].float()
    if case["op"] in ("w4", "w4_gated"):
        P = [A @ _dequantize(*w, case["group"], case["K"]).t() for w in s["W4"]]
        return (P[0] if case["op"] == "w4" else _act(P[0], case["act"]) * P[1]).to(dt)
    G, U = s["G"].float(), s["U"].float()
    g, u = A @ G.t(), A @ U.t()
    if case["op"] == "gated":
        return (_act(g, case["act"]) * u).to(dt)
    dH = s["dH"].float()
    dg = dH * u * _act_slope(g, case["act"])
    du = dH * _act(g, case["act"])
    return {"dA": (dg @ G + du @ U).to(dt), "dG": (dg.t() @ A).to(dt), "dU": (du.t() @ A).to(dt)}


# ------------------------------------------------------------ the operators

def run(state):
    if not own:
        return _plain(state)
    import dense_gemm_preshuffle_gb300 as gp
    case = state["case"]
    if case["op"] == "gated":
        return gp.gated_matmul(state["A"], state["G"], state["U"], act=case["act"])
    if case["op"] == "gated_back":
        dA, dG, dU = gp.gated_matmul_backward(state["A"], state["G"], state["U"], state["dH"], act=case["act"])
        return {"dA": dA, "dG": dG, "dU": dU}
    if case["op"] == "w4":
        return gp.matmul_w4g(state["A"], state["packed"][0], b_constant=True)
    return gp.matmul_w4g_gated(state["A"], state["packed"][0], state["packed"][1], act=case["act"], b_constant=True)


def work(case):
    M, N, K = case["M"], case["N"], case["K"]
    if case["op"] == "gated":
        return {"bytes": 2 * (M * K + 2 * N * K + M * N), "flops": 4 * M * N * K}
    if case["op"] == "gated_back":
        # read A, G, U, dH; write dA, dG, dU.  Six products: two recomputed, two for dA, two for the weights.
        return {"bytes": 2 * (2 * M * K + 4 * N * K + M * N), "flops": 12 * M * N * K}
    groups = (K + case["group"] - 1) // case["group"]
    weights = N * K // 2 + N * groups * (3 if case["zeros"] else 2)
    count = 1 if case["op"] == "w4" else 2
    return {"bytes": count * weights + 2 * (M * K + M * N), "flops": 2 * count * M * N * K}


# ------------------------------------------------------------ the definition in 64 bits

def _erf64(x):
    return torch.special.erf(x)


def exact(case, seed):
    s = prepare(case, seed)
    A = s["A"].to(torch.float64)

    def act_of(x):
        if case["act"] == "silu":
            return x * torch.sigmoid(x)
        if case["act"] == "gelu":
            return x * (1.0 + _erf64(x / np.sqrt(2.0))) / 2.0
        return torch.clamp(x, min=0.0)

    def slope_of(x):
        if case["act"] == "silu":
            t = torch.sigmoid(x)
            return t + x * t * (1.0 - t)
        if case["act"] == "gelu":
            return (1.0 + _erf64(x / np.sqrt(2.0))) / 2.0 + x * torch.exp(-x * x / 2.0) / np.sqrt(2.0 * np.pi)
        return torch.where(x > 0, 1.0, 0.0).to(torch.float64)

    if case["op"] in ("w4", "w4_gated"):
        products = []
        for codes, scales, zeros in s["W4"]:
            out = torch.empty((case["M"], case["N"]), dtype=torch.float64, device="cuda")
            for n0 in range(0, case["N"], 8192):  # rows at a time: the weights in 64 bits are large
                c = codes[n0:n0 + 8192].to(torch.int64)
                w = torch.empty((c.shape[0], case["K"]), dtype=torch.float64, device="cuda")
                w[:, 0::2] = (c % 16).to(torch.float64)
                w[:, 1::2] = torch.div(c, 16, rounding_mode="floor").to(torch.float64)
                for j in range(scales.shape[1]):
                    part = w[:, j * case["group"]:(j + 1) * case["group"]]
                    part -= 8.0 if zeros is None else zeros[n0:n0 + 8192, j:j + 1].to(torch.float64)
                    part *= scales[n0:n0 + 8192, j:j + 1].to(torch.float64)
                out[:, n0:n0 + 8192] = A @ w.T
            products.append(out)
        return products[0] if case["op"] == "w4" else act_of(products[0]) * products[1]
    G, U = s["G"].to(torch.float64), s["U"].to(torch.float64)
    g, u = A @ G.T, A @ U.T
    if case["op"] == "gated":
        return act_of(g) * u
    dH = s["dH"].to(torch.float64)
    dg, du = dH * u * slope_of(g), dH * act_of(g)
    return {"dA": dg @ G + du @ U, "dG": dg.T @ A, "dU": du.T @ A}
