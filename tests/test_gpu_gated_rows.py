"""The gated products for tens to a few hundred tokens, whose kernel has the
weights as the MMA's rows: the shapes that go to it, every form of ragged
shape with it forced, and its bounded waits."""
import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest
import torch

import dense_gemm_preshuffle_gb300 as gp
from oracle import ffn

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_gemm_preshuffle_gb300 import build
    build.build()
    gp.load_library()


def f64(t):
    return t.double().cpu().numpy()


def rows(r, c, dtype, seed, scale=1.0, pad=8):
    """[r, c] with NaN behind every row's end."""
    buf = torch.full((r, (c + 7) // 8 * 8 + pad), float("nan"), dtype=TYPES[dtype], device="cuda")
    buf[:, :c] = torch.from_numpy(np.random.default_rng(seed).standard_normal((r, c)) * scale).to(TYPES[dtype]).cuda()
    return buf[:, :c]


def check(M, N, K, dtype, act, seed=0, backward=True):
    A, dH = rows(M, K, dtype, seed + 1), rows(M, N, dtype, seed + 2)
    G, U = (rows(N, K, dtype, seed + s, K ** -0.5) for s in (3, 4))
    buf = torch.full((M, (N + 7) // 8 * 8 + 8), float("nan"), dtype=TYPES[dtype], device="cuda")
    ops = [f64(x) for x in (A, G, U)]
    gp.gated_matmul(A, G, U, act=act, out=buf[:, :N])
    want, bound = ffn.gated_bound(*ops, act, dtype)
    assert (np.abs(f64(buf[:, :N]) - want) <= bound).all(), (M, N, K, dtype, act)
    assert torch.isnan(buf[:, N:]).all()
    assert torch.equal(gp.gated_matmul(A, G, U, act=act, b_constant=True), buf[:, :N])
    if backward:
        want, bounds = ffn.gated_backward_bound(*ops, f64(dH), act, dtype)
        for o, w, b in zip(gp.gated_matmul_backward(A, G, U, dH, act=act), want, bounds):
            assert (np.abs(f64(o) - w) <= b).all(), (M, N, K, dtype, act)


@pytest.mark.parametrize("M,N,K", [(16, 7168, 1030), (42, 1370, 5627), (64, 500, 4096), (97, 2041, 4099), (130, 4097, 770),
                                   (200, 301, 6001), (256, 1000, 2050), (33, 16400, 200)])
@pytest.mark.parametrize("dtype,act", [("bf16", "silu"), ("fp16", "gelu")])
def test_tens_of_tokens(M, N, K, dtype, act):
    check(M, N, K, dtype, act, backward=N * K < 4_000_000)
    assert gp.gemm_last_device_status() == 0


def test_a_row_keeps_its_nan():
    A = rows(70, 4096, "bf16", 5)
    G, U = (rows(1500, 4096, "bf16", s, 1 / 64) for s in (6, 7))
    plain = gp.gated_matmul(A, G, U)
    A[1], A[2, 5] = 0, float("nan")
    got = gp.gated_matmul(A, G, U)
    assert not got[1].any() and torch.isnan(got[2]).all()
    keep = [i for i in range(70) if i not in (1, 2)]
    assert torch.equal(got[keep], plain[keep])


def test_chain_on_a_side_stream():
    A = rows(48, 2048, "bf16", 8, pad=0)
    G, U = (rows(2048, 2048, "bf16", s, 1 / 32) for s in (9, 10))
    want = A
    for _ in range(6):
        want = gp.gated_matmul(want, G, U)
    torch.cuda.synchronize()
    side, got = torch.cuda.Stream(), A
    with torch.cuda.stream(side):
        for i in range(6):
            got = gp.gated_matmul(got, G, U, b_constant=bool(i % 2))
    side.synchronize()
    assert torch.isfinite(want).all() and torch.equal(got, want)


HEAD = textwrap.dedent("""
    import sys, time
    sys.path.insert(0, {root!r})
    sys.path.insert(0, {tests!r})
    import dense_gemm_preshuffle_gb300 as gp
    import test_gpu_gated_rows as t
    gp.load_library()
""").format(root=ROOT, tests=os.path.dirname(os.path.abspath(__file__)))

FORMS = HEAD + textwrap.dedent("""
    for i, (M, N, K) in enumerate([(1, 1, 1), (1, 100, 72), (3, 513, 640), (9, 64, 1000), (16, 31, 65), (17, 250, 129),
                                   (40, 700, 64), (64, 128, 2048), (65, 129, 2500), (128, 9800, 70), (200, 300, 320),
                                   (255, 40, 4090), (256, 260, 65), (48, 24000, 130)]):
        t.check(M, N, K, ("bf16", "fp16")[i % 2], ("silu", "gelu", "relu")[i % 3], seed=i, backward=N < 9000)
    assert gp.gemm_last_device_status() == 0
    print("all shapes right")
""")

FAULT = HEAD + textwrap.dedent("""
    A = t.rows(M, K, "bf16", 1)
    G, U = (t.rows(N, K, "bf16", s, K ** -0.5) for s in (2, 3))
    t.torch.cuda.synchronize()
    assert gp.gemm_last_device_status() == 0
    gp.gemm_debug_skip_load(2)
    t0 = time.time()
    gp.gated_matmul(A, G, U, b_constant=b_constant)
    st = gp.gemm_last_device_status()
    assert st == 6, f"expected GP_ERR_DEVICE_TIMEOUT, got {st}"
    assert time.time() - t0 < 20
    t.check(M, N, K, "bf16", "silu")
    assert gp.gemm_last_device_status() == 0
    print("next calls ok")
""")


def child(code, **env):
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, **env), capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


def test_every_shape():
    """A child process, because the choice is read once."""
    assert "all shapes right" in child(FORMS, GP_GATED_STREAM="2")


@pytest.mark.parametrize("M,N,K,b_constant", [(40, 1500, 512, False), (64, 300, 4096, True), (32, 12000, 256, False)])
def test_timeout_is_reported_and_the_context_survives(M, N, K, b_constant):
    """A stage's copies left out, as the bounded waits of the other kernels are tested."""
    sizes = f"M, N, K, b_constant = {M}, {N}, {K}, {b_constant}\n"
    assert "next calls ok" in child(sizes + FAULT, GP_GATED_STREAM="2", GP_WAIT_LIMIT_MS="200")


CHUNKS = HEAD + textwrap.dedent("""
    for i, (M, N, K) in enumerate([(257, 500, 4097), (300, 1000, 2000), (513, 90, 1500), (700, 831, 130),
                                   (1024, 250, 640), (1001, 3000, 65)]):
        t.check(M, N, K, ("bf16", "fp16")[i % 2], ("silu", "gelu", "relu")[i % 3], seed=i)
    assert gp.gemm_last_device_status() == 0
    print("all shapes right")
""")


@pytest.mark.parametrize("form", ["2", ""])
def test_more_tokens_than_one_unit_takes(form):
    assert "all shapes right" in child(CHUNKS, GP_GATED_STREAM=form)
