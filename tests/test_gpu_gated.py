"""Gated products and their gradients on the GPU, against the 64-bit
definitions and the error bounds of oracle.ffn: every element of every
output, outputs filled with NaN first, rows padded with NaN."""
import numpy as np
import pytest
import torch

import dense_gemm_preshuffle_gb300 as gp
from oracle import ffn

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_gemm_preshuffle_gb300 import build
    build.build()
    gp.load_library()
    yield
    assert gp.gemm_last_device_status() == 0


def rows(values, dtype, pad=0):
    """A device copy whose rows start on 16-byte boundaries, `pad` * 8 spare
    elements apart, everything outside the rows NaN."""
    r, c = values.shape
    ld = (c + 7) // 8 * 8 + 8 * pad
    buf = torch.full((r, ld), float("nan"), dtype=TYPES[dtype], device="cuda")
    buf[:, :c] = torch.from_numpy(values).to(TYPES[dtype]).cuda()
    return buf[:, :c]


def f64(t):
    return t.double().cpu().numpy()


def untouched(view):
    """The spare elements between the rows of `view` are still NaN."""
    whole = view._base
    return view.shape[1] == whole.shape[1] or bool(torch.isnan(whole[:, view.shape[1]:]).all())


def operands(M, N, K, dtype, seed=0, pad=1, scale=1.0):
    rng = np.random.default_rng(seed + 1000 * M + 10 * N + K)
    A = rows(rng.standard_normal((M, K)) * scale, dtype, pad)
    G = rows(rng.standard_normal((N, K)) / np.sqrt(K), dtype, pad)
    U = rows(rng.standard_normal((N, K)) / np.sqrt(K), dtype, pad + 1)
    dH = rows(rng.standard_normal((M, N)), dtype, pad)
    return A, G, U, dH


def empty(r, c, dtype, pad=1):
    return rows(np.full((r, c), np.nan), dtype, pad)


def within(got, want, bound):
    got = f64(got)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {want[bad][0]} +- {bound[bad][0]}")


FORWARD = [(1, 1, 1), (1, 8, 8), (1, 130, 72), (2, 257, 64), (3, 129, 1093), (7, 64, 40), (8, 200, 136), (9, 256, 512),
           (16, 384, 320), (17, 129, 65), (31, 100, 257), (33, 128, 128), (64, 255, 193), (65, 256, 64), (127, 300, 72),
           (128, 128, 2048), (129, 1000, 63), (200, 137, 1024), (255, 257, 129), (256, 256, 256), (257, 513, 100),
           (300, 128, 4097), (513, 640, 200), (1000, 72, 520)]


@pytest.mark.parametrize("M,N,K", FORWARD)
@pytest.mark.parametrize("dtype,act", [("bf16", "silu"), ("fp16", "gelu"), ("bf16", "relu")])
def test_forward(M, N, K, dtype, act):
    A, G, U, _ = operands(M, N, K, dtype)
    out = empty(M, N, dtype)
    got = gp.gated_matmul(A, G, U, act=act, out=out)
    assert got is out
    within(out, *ffn.gated_bound(f64(A), f64(G), f64(U), act, dtype))
    assert untouched(out)


@pytest.mark.parametrize("M,N,K", [(2, 500, 4100), (11, 300, 3331), (30, 700, 5000), (60, 200, 4097)])
def test_few_tokens_and_long_sums(M, N, K):
    """Rows of weights too few to fill the GPU: four blocks share each 16."""
    A, G, U, dH = operands(M, N, K, "bf16", seed=8)
    first = gp.gated_matmul(A, G, U)
    within(first, *ffn.gated_bound(f64(A), f64(G), f64(U), "silu", "bf16"))
    for _ in range(10):
        assert torch.equal(gp.gated_matmul(A, G, U, b_constant=True), first)
    want, bounds = ffn.gated_backward_bound(f64(A), f64(G), f64(U), f64(dH), "silu", "bf16")
    for o, w, b in zip(gp.gated_matmul_backward(A, G, U, dH), want, bounds):
        within(o, w, b)


BACKWARD = [(1, 1, 1), (1, 200, 72), (2, 64, 257), (5, 129, 65), (17, 130, 136), (64, 100, 300), (127, 257, 129),
            (128, 256, 256), (130, 65, 1030), (255, 511, 120), (257, 300, 257), (300, 1100, 64), (700, 129, 200),
            (1025, 72, 530)]


@pytest.mark.parametrize("M,N,K", BACKWARD)
@pytest.mark.parametrize("dtype,act", [("bf16", "silu"), ("fp16", "gelu"), ("fp16", "relu")])
def test_backward(M, N, K, dtype, act):
    A, G, U, dH = operands(M, N, K, dtype, seed=1)
    out = (empty(M, K, dtype), empty(N, K, dtype), empty(N, K, dtype, 2))
    nbytes = gp.gemm_gated_backward_workspace_bytes(M, N, K)
    ws = torch.full((nbytes + 64,), 255, dtype=torch.uint8, device="cuda")  # NaN as either type
    gp.gated_matmul_backward(A, G, U, dH, act=act, out=out, workspace=ws[:nbytes])
    want, bounds = ffn.gated_backward_bound(f64(A), f64(G), f64(U), f64(dH), act, dtype)
    for o, w, b in zip(out, want, bounds):
        within(o, w, b)
        assert untouched(o)
    assert bool((ws[nbytes:] == 255).all())  # nothing past the stated size


@pytest.mark.parametrize("M,N,K", [(300, 500, 4000), (260, 1001, 1100), (520, 196, 2111), (129, 2, 5000)])
@pytest.mark.parametrize("dtype,act", [("bf16", "silu"), ("fp16", "gelu"), ("bf16", "relu")])
def test_backward_long_sums(M, N, K, dtype, act):
    """Few tiles and a long sum: the gates' own products are split along it too."""
    test_backward(M, N, K, dtype, act)
    operand = operands(M, N, K, dtype, seed=1)
    first = gp.gated_matmul_backward(*operand, act=act)
    for need in ({}, {"need_dA": False}, {"need_dW": False}):
        again = gp.gated_matmul_backward(*operand, act=act, **need)
        assert all(x is None or torch.equal(x, y) for x, y in zip(again, first))


@pytest.mark.parametrize("need_dA,need_dW", [(True, False), (False, True)])
def test_backward_in_parts(need_dA, need_dW):
    A, G, U, dH = operands(70, 190, 130, "bf16", seed=2)
    whole = gp.gated_matmul_backward(A, G, U, dH)
    part = gp.gated_matmul_backward(A, G, U, dH, need_dA=need_dA, need_dW=need_dW)
    assert (part[0] is None) != need_dA and (part[1] is None) != need_dW and (part[2] is None) != need_dW
    for w, p in zip(whole, part):
        assert p is None or torch.equal(w, p)


@pytest.mark.parametrize("M,N,K", [(24, 40, 56), (130, 72, 48)])
def test_gradients_against_differences(M, N, K):
    """The derivative of the 64-bit loss along random directions."""
    ops = operands(M, N, K, "fp16", seed=3)
    A, G, U, dH = (f64(t) for t in ops)
    grads = [f64(t) for t in gp.gated_matmul_backward(*ops, act="gelu")]
    _, bounds = ffn.gated_backward_bound(A, G, U, dH, "gelu", "fp16")
    rng = np.random.default_rng(9)
    h = 1e-4
    for i in range(3):
        v = rng.standard_normal((A, G, U)[i].shape)
        shifted = [[x + s * h * v if j == i else x for j, x in enumerate((A, G, U))] for s in (1, -1)]
        num = sum(s * (ffn.gated(*x, "gelu") * dH).sum() for s, x in zip((1, -1), shifted)) / (2 * h)
        # third derivatives times h^2 / 6 stay far below the elements' own bounds
        assert abs(num - (grads[i] * v).sum()) <= (bounds[i] * np.abs(v)).sum()


@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
@pytest.mark.parametrize("M", [4, 300])
def test_saturated_gates(act, M):
    """Gates far out on both sides: no infinities of an exponential get through."""
    A, G, U, dH = operands(M, 140, 64, "bf16", seed=4, scale=120.0)
    within(gp.gated_matmul(A, G, U, act=act), *ffn.gated_bound(f64(A), f64(G), f64(U), act, "bf16"))
    want, bounds = ffn.gated_backward_bound(f64(A), f64(G), f64(U), f64(dH), act, "bf16")
    for o, w, b in zip(gp.gated_matmul_backward(A, G, U, dH, act=act), want, bounds):
        within(o, w, b)


@pytest.mark.parametrize("M", [3, 200])
def test_masked_rows(M):
    """Rows of A and dH that a mask zeroed, and a NaN that stays in its own row."""
    A, G, U, dH = operands(M, 150, 80, "bf16", seed=5)
    A[0] = 0
    dH[1] = 0
    H = gp.gated_matmul(A, G, U)
    dA, dG, dU = gp.gated_matmul_backward(A, G, U, dH)
    assert not H[0].any() and not dA[1].any()
    within(H, *ffn.gated_bound(f64(A), f64(G), f64(U), "silu", "bf16"))
    (wA, _, _), (bA, _, _) = ffn.gated_backward_bound(f64(A), f64(G), f64(U), f64(dH), "silu", "bf16")
    within(dA, wA, bA)
    A[2, 7] = float("nan")
    again = gp.gated_matmul(A, G, U)
    assert torch.isnan(again[2]).all()
    keep = [i for i in range(M) if i != 2]
    assert torch.equal(again[keep], H[keep])
    dA2 = gp.gated_matmul_backward(A, G, U, dH, need_dW=False)[0]
    assert torch.isnan(dA2[2]).all() and torch.equal(dA2[keep], dA[keep])


def test_empty_sizes():
    z = dict(dtype=torch.bfloat16, device="cuda")
    w = torch.randn((24, 16), **z)
    assert gp.gated_matmul(torch.empty((0, 16), **z), w, w).shape == (0, 24)
    assert gp.gated_matmul(torch.randn((3, 16), **z), w[:0], w[:0]).shape == (3, 0)
    e = torch.empty((24, 0), **z)
    out = torch.full((3, 24), float("nan"), **z)
    gp.gated_matmul(torch.empty((3, 0), **z), e, e, out=out)
    assert not out.any() and not torch.isnan(out).any()
    dA, dG, dU = gp.gated_matmul_backward(torch.empty((0, 16), **z), w, w, torch.empty((0, 24), **z))
    assert dA.shape == (0, 16) and not dG.any() and not dU.any()
    dA, dG, dU = gp.gated_matmul_backward(torch.randn((3, 16), **z), w[:0], w[:0], torch.empty((3, 0), **z))
    assert not dA.any() and dG.shape == (0, 16)


@pytest.mark.parametrize("M,N,K", [(5, 300, 256), (300, 520, 256), (130, 260, 2100)])
def test_repeats_are_bit_identical(M, N, K):
    A, G, U, dH = operands(M, N, K, "bf16", seed=6)
    first = (gp.gated_matmul(A, G, U), *gp.gated_matmul_backward(A, G, U, dH))
    for _ in range(10):
        again = (gp.gated_matmul(A, G, U), *gp.gated_matmul_backward(A, G, U, dH))
        assert all(torch.equal(x, y) for x, y in zip(first, again))


@pytest.mark.parametrize("M", [6, 260])
def test_side_stream_and_chained_calls(M):
    """A chain of dependent calls on a stream of its own: each reads what the one before wrote."""
    A, G, U, _ = operands(M, 256, 256, "bf16", seed=7, pad=0)
    want = A
    for _ in range(6):
        want = gp.gated_matmul(want, G, U)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = A
    with torch.cuda.stream(side):
        for i in range(6):
            got = gp.gated_matmul(got, G, U, b_constant=bool(i % 2))
    side.synchronize()
    assert torch.equal(got, want)


def test_rows_past_32_bit_offsets():
    """Rows further than 2^32 elements from the first."""
    M, ld, K, N = 70000, 65544, 40, 24
    A = torch.empty((M, ld), dtype=torch.bfloat16, device="cuda")[:, :K]
    gen = torch.Generator(device="cuda").manual_seed(1)
    A.copy_(torch.randn((M, K), generator=gen, device="cuda"))
    G, U = (torch.randn((N, K), generator=gen, device="cuda").div_(6).to(torch.bfloat16) for _ in range(2))
    H = torch.empty((M, ld), dtype=torch.bfloat16, device="cuda")[:, :N]
    gp.gated_matmul(A, G, U, out=H)
    for part in (slice(0, 300), slice(M - 300, M)):
        within(H[part], *ffn.gated_bound(f64(A[part]), f64(G), f64(U), "silu", "bf16"))


def test_many_drawn_shapes():
    rng = np.random.default_rng(11)
    for i in range(24):
        M, N, K = (int(np.exp(rng.uniform(0, np.log(hi)))) for hi in (900, 700, 700))
        dtype, act = ("bf16", "fp16")[i % 2], ("silu", "gelu", "relu")[i % 3]
        A, G, U, dH = operands(M, N, K, dtype, seed=20 + i, pad=i % 3)
        within(gp.gated_matmul(A, G, U, act=act), *ffn.gated_bound(f64(A), f64(G), f64(U), act, dtype))
        want, bounds = ffn.gated_backward_bound(f64(A), f64(G), f64(U), f64(dH), act, dtype)
        for o, w, b in zip(gp.gated_matmul_backward(A, G, U, dH, act=act), want, bounds):
            within(o, w, b)


def test_refusals():
    z = dict(dtype=torch.bfloat16, device="cuda")
    A, W = torch.zeros((4, 64), **z), torch.zeros((32, 64), **z)
    bad = [
        lambda: gp.gated_matmul(A, W, W.half()),                      # two types
        lambda: gp.gated_matmul(A.float(), W.float(), W.float()),     # not a 16-bit float
        lambda: gp.gated_matmul(A, W, W[:, :56]),                     # shapes
        lambda: gp.gated_matmul(A, W, W, act="tanh"),
        lambda: gp.gated_matmul(A, W, W, out=torch.empty((4, 40), **z)),
        lambda: gp.gated_matmul(A, torch.zeros((64, 32), **z).t(), W),  # rows not contiguous
        lambda: gp.gated_matmul_backward(A, W, W, torch.zeros((4, 31), **z)),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    odd = torch.zeros((4, 65), **z)
    for call, code in [
        (lambda: gp.gated_matmul(odd[:, :64], W, W), 3),              # a pitch of 65
        (lambda: gp.gated_matmul(torch.zeros(4 * 64 + 8, **z)[4:4 + 256].view(4, 64), W, W), 4),
        (lambda: gp.gated_matmul_backward(A, W, W, torch.zeros((4, 32), **z),
                                          workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), 3),
    ]:
        with pytest.raises(gp.GemmError) as e:
            call()
        assert e.value.code == code
