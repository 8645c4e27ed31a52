"""Plain 64-bit definitions of the feed-forward operators, with error bounds.

Test infrastructure only, as the rest of this package: numpy in fp64, no code
shared with the CUDA path.

    gated        H = act(A G^T) * (A U^T)
    gradients    of sum(H * dH):  dg = dH u act'(g), du = dH act(g),
                 dA = dg G + du U, dG = dg^T A, dU = du^T A
    w4g          W[n, k] = (q[n, k] - z[n, k // group]) * s[n, k // group]

The bounds follow from the number formats alone.  UNIT is the largest
relative error of one rounding to the type.  An fp32 sum of n products is
taken to be within n * 2^-23 of the sum of their absolute values: one ulp
(the tensor cores truncate where scalar code rounds) per addition.  EVAL is
the relative error of evaluating an activation in fp32, including its
exponential and reciprocal, with |v| times it again for the argument of the
exponential.
"""
from __future__ import annotations

import math
from typing import Optional

import numpy as np

UNIT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
SMALLEST = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}  # half the spacing of the smallest values
SUM_STEP = 2.0 ** -23
EVAL = 2.0 ** -20

_erf = np.frompyfunc(math.erf, 1, 1)


def erf(x: np.ndarray) -> np.ndarray:
    return _erf(x).astype(np.float64)


def _sigmoid(v: np.ndarray) -> np.ndarray:
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def act(v: np.ndarray, name: str) -> np.ndarray:
    if name == "relu":
        return np.maximum(v, 0.0)
    if name == "silu":
        return v * _sigmoid(v)
    if name == "gelu":
        return 0.5 * v * (1.0 + erf(v / math.sqrt(2.0)))
    raise ValueError(name)


def act_slope(v: np.ndarray, name: str) -> np.ndarray:
    if name == "relu":
        return (v > 0).astype(np.float64)
    if name == "silu":
        s = _sigmoid(v)
        return s * (1.0 + v * (1.0 - s))
    if name == "gelu":
        return 0.5 * (1.0 + erf(v / math.sqrt(2.0))) + v * np.exp(-0.5 * v * v) / math.sqrt(2.0 * math.pi)
    raise ValueError(name)


# |act''| is at most 1/2 for SiLU and 2 / sqrt(2 pi) for GELU, |act'| at most 1.13
CURVATURE = {"relu": 0.0, "silu": 0.5, "gelu": 0.8}
STEEPEST = 1.13


def gated(A: np.ndarray, G: np.ndarray, U: np.ndarray, name: str):
    """H in fp64."""
    return act(A @ G.T, name) * (A @ U.T)


def _pre(A, G, U):
    K = A.shape[1]
    aA = np.abs(A)
    g, u = A @ G.T, A @ U.T
    eg = K * SUM_STEP * (aA @ np.abs(G).T)
    eu = K * SUM_STEP * (aA @ np.abs(U).T)
    return g, u, eg, eu


def gated_bound(A, G, U, name: str, dtype: str):
    """(H, the largest error of each element of a result in `dtype`)."""
    g, u, eg, eu = _pre(A, G, U)
    return _gate(g, u, eg, eu, name, dtype)


def _gate(g, u, eg, eu, name, dtype):
    a = act(g, name)
    ea = STEEPEST * eg + EVAL * np.abs(g)
    H = a * u
    e = ea * np.abs(u) + np.abs(a) * eu + ea * eu
    return H, e + UNIT[dtype] * (np.abs(H) + e) + SMALLEST[dtype]


def gated_backward(A, G, U, dH, name: str):
    """(dA, dG, dU) in fp64."""
    g, u = A @ G.T, A @ U.T
    dg, du = dH * u * act_slope(g, name), dH * act(g, name)
    return dg @ G + du @ U, dg.T @ A, du.T @ A


def gated_backward_bound(A, G, U, dH, name: str, dtype: str):
    """((dA, dG, dU), their bounds): dg and du are rounded to `dtype` before the last products."""
    g, u, eg, eu = _pre(A, G, U)
    d = np.abs(dH)
    s, a = act_slope(g, name), act(g, name)
    es = CURVATURE[name] * eg + EVAL * (1.0 + np.abs(g))
    if name == "relu":  # within its error of 0, the slope may be either
        es = es + (np.abs(g) <= eg)
    dg, du = dH * u * s, dH * a
    edg = d * (np.abs(u) * es + np.abs(s) * eu + es * eu)
    edu = d * (STEEPEST * eg + EVAL * np.abs(g))
    edg = edg + UNIT[dtype] * (np.abs(dg) + edg) + SMALLEST[dtype]
    edu = edu + UNIT[dtype] * (np.abs(du) + edu) + SMALLEST[dtype]

    def done(value, e):
        return e + UNIT[dtype] * (np.abs(value) + e) + SMALLEST[dtype]

    M, N = g.shape
    aA, aG, aU = np.abs(A), np.abs(G), np.abs(U)
    adg, adu = np.abs(dg) + edg, np.abs(du) + edu
    dA, dG, dU = dg @ G + du @ U, dg.T @ A, du.T @ A
    bA = edg @ aG + edu @ aU + 2 * N * SUM_STEP * (adg @ aG + adu @ aU)
    bG = edg.T @ aA + M * SUM_STEP * (adg.T @ aA)
    bU = edu.T @ aA + M * SUM_STEP * (adu.T @ aA)
    return (dA, dG, dU), (done(dA, bA), done(dG, bG), done(dU, bU))


# ------------------------------------------------------------------ 4-bit weights

def w4g_codes(codes: np.ndarray) -> np.ndarray:
    """uint8 [N, K/2] -> int64 [N, K], the even-k code in the low nibble."""
    out = np.empty((codes.shape[0], codes.shape[1] * 2), dtype=np.int64)
    out[:, 0::2] = codes & 15
    out[:, 1::2] = codes >> 4
    return out


def w4g_dequantize(codes: np.ndarray, scales: np.ndarray, zeros: Optional[np.ndarray], group: int) -> np.ndarray:
    q = w4g_codes(codes).astype(np.float64)
    j = np.arange(q.shape[1]) // group
    z = 8.0 if zeros is None else zeros.astype(np.float64)[:, j]
    return (q - z) * scales.astype(np.float64)[:, j]


def w4g_sum_bound(A, codes, scales, zeros, group: int) -> np.ndarray:
    """Error bound of the fp32 sums of A . W^T.  Each group is summed over
    codes offset by 128 (so that a code is its own 16-bit float), the offset
    and the zero point are taken off as (128 + z) times the group's sum of A:
    every term of both is at most 144 |a|.  The groups are then added."""
    K = A.shape[1]
    groups = scales.shape[1]
    aA = np.abs(A)
    sums = np.stack([aA[:, j * group:(j + 1) * group].sum(axis=1) for j in range(groups)], axis=1)
    in_group = 3 * group * SUM_STEP * 144.0 * (sums @ np.abs(scales).T)
    total = np.abs(A) @ np.abs(w4g_dequantize(codes, scales, zeros, group)).T
    return in_group + (groups + 64) * SUM_STEP * (total + in_group)


def w4g_bound(A, weights, group: int, dtype: str, name: Optional[str] = None):
    """(C, bound) of the product with one (codes, scales, zeros), or of the gated pair."""
    P = [A @ w4g_dequantize(*w, group).T for w in weights]
    E = [w4g_sum_bound(A, *w, group) for w in weights]
    if name is not None:
        return _gate(P[0], P[1], E[0], E[1], name, dtype)
    return P[0], E[0] + UNIT[dtype] * (np.abs(P[0]) + E[0]) + SMALLEST[dtype]


def w4g_pack(codes: np.ndarray, scales_bits: np.ndarray, zeros: Optional[np.ndarray], group: int) -> np.ndarray:
    """The packed buffer, element by element from the documented layout."""
    N, K = codes.shape[0], codes.shape[1] * 2
    q = w4g_codes(codes)
    kb, rt, gpb = -(-K // 128), -(-N // 64) * 4, 128 // group
    size = 1024 + (32 if zeros is None else 48) * gpb
    out = np.zeros((rt * kb, size), dtype=np.uint8)
    place = [0, 16, 4, 20, 8, 24, 12, 28]
    for n in range(N):
        r, h, g = n // 16, n // 8 % 2, n % 8
        for k0 in range(0, K, 8):
            c, i, t = k0 // 128, k0 % 128 // 32, k0 % 32 // 8
            w = sum(int(q[n, k0 + e]) << place[e] for e in range(8))
            at = (h * 32 + 4 * g + t) * 16 + 4 * i
            out[r * kb + c, at:at + 4] = np.frombuffer(w.to_bytes(4, "little"), dtype=np.uint8)
        for j in range(scales_bits.shape[1]):
            at = (g * gpb + j % gpb) * 2 + h
            block = out[r * kb + j // gpb, 1024:]
            block[2 * at:2 * at + 2] = np.frombuffer(int(scales_bits[n, j]).to_bytes(2, "little"), dtype=np.uint8)
            if zeros is not None:
                block[32 * gpb + at] = zeros[n, j]
    return out.reshape(-1)
