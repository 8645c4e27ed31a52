"""Products with 4-bit weights and more rows of A than one pass of the
streaming kernel takes: the shapes that go to the tile kernel, either kernel on
every shape, and the tile kernel's bounded waits."""
import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest
import torch

import dense_gemm_preshuffle_gb300 as gp
from oracle import ffn

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


def weights(N, K, group, zeros, dtype, seed):
    rng = np.random.default_rng(seed)
    groups = -(-K // group)
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    scales = torch.from_numpy((rng.random((N, groups)) + 0.5) / np.sqrt(K) / 4).to(TYPES[dtype]).cuda()
    zp = rng.integers(0, 16, (N, groups), dtype=np.uint8) if zeros else None
    W = gp.preshuffle_w4g(torch.from_numpy(codes).cuda(), scales, group,
                          zeros=None if zp is None else torch.from_numpy(zp).cuda())
    return (codes, f64(scales), zp), W


def rows(M, K, dtype, seed, pad=8):
    buf = torch.full((M, K + pad), float("nan"), dtype=TYPES[dtype], device="cuda")
    buf[:, :K] = torch.from_numpy(np.random.default_rng(seed).standard_normal((M, K))).to(TYPES[dtype]).cuda()
    return buf[:, :K]


def check(M, N, K, group, zeros, dtype, scale_type, gated, seed=0):
    w, W = weights(N, K, group, zeros, scale_type, seed + 1)
    A = rows(M, K, dtype, seed + 2)
    buf = torch.full((M, N + 5), float("nan"), dtype=TYPES[dtype], device="cuda")
    out = buf[:, :N]
    if gated:
        u, U = weights(N, K, group, zeros, scale_type, seed + 3)
        gp.matmul_w4g_gated(A, W, U, act="silu", out=out)
        want, bound = ffn.w4g_bound(f64(A), [w, u], group, dtype, "silu")
    else:
        gp.matmul_w4g(A, W, out=out)
        want, bound = ffn.w4g_bound(f64(A), [w], group, dtype)
    bad = ~(np.abs(f64(out) - want) <= bound)
    assert not bad.any(), (M, N, K, group, zeros, dtype, gated, int(bad.sum()), np.argwhere(bad)[0])
    assert torch.isnan(buf[:, N:]).all()
    again = gp.matmul_w4g_gated(A, W, U, act="silu") if gated else gp.matmul_w4g(A, W, b_constant=True)
    assert torch.equal(again, out)


# the last block of K half used, K past a step's 256 values, columns past the
# last 64 and 128, one to several units a CTA, a cluster to a unit
LARGE = [(17, 9000, 4128), (32, 2500, 8192), (33, 4097, 2976), (64, 21000, 544), (70, 5119, 1056), (200, 3001, 2048),
         (130, 1000, 7200)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", LARGE)
@pytest.mark.parametrize("group,zeros,dtype,scale_type,gated", [
    (128, False, "bf16", "bf16", False), (64, True, "fp16", "fp16", True), (32, True, "bf16", "fp16", False),
    (128, True, "fp16", "bf16", True), (32, False, "fp16", "fp16", False)])
def test_many_rows(M, N, K, group, zeros, dtype, scale_type, gated):
    check(M, N, K, group, zeros, dtype, scale_type, gated)
    assert gp.gemm_last_device_status() == 0


@pytest.mark.gpu
def test_a_row_keeps_its_nan():
    _, W = weights(9000, 4096, 128, False, "bf16", 5)
    A = rows(40, 4096, "bf16", 6)
    plain = gp.matmul_w4g(A, W)
    A[1], A[2, 5], A[39, 4095] = 0, float("nan"), float("inf")
    got = gp.matmul_w4g(A, W)
    assert not got[1].any() and torch.isnan(got[2]).all() and not torch.isfinite(got[39]).any()
    keep = [i for i in range(40) if i not in (1, 2, 39)]
    assert torch.equal(got[keep], plain[keep])


@pytest.mark.gpu
def test_chain_on_a_side_stream():
    """Each call reads what the one before it wrote; packed weights may be read early."""
    _, W = weights(4096, 4096, 128, True, "bf16", 7)
    A = rows(64, 4096, "bf16", 8, pad=0)
    want = A
    for _ in range(6):
        want = gp.matmul_w4g(want, W)
    torch.cuda.synchronize()
    side, got = torch.cuda.Stream(), A
    with torch.cuda.stream(side):
        for i in range(6):
            got = gp.matmul_w4g(got, W, b_constant=bool(i % 2))
    side.synchronize()
    assert torch.isfinite(want).all() and torch.equal(got, want)


FORMS = textwrap.dedent("""
    import sys
    sys.path.insert(0, {root!r})
    sys.path.insert(0, {tests!r})
    import dense_gemm_preshuffle_gb300 as gp
    import test_gpu_w4g_tiles as t
    gp.load_library()
    shapes = [(1, 1, 32), (1, 300, 4096), (3, 129, 96), (8, 64, 8192), (16, 65, 128), (17, 1, 32), (20, 200, 2080),
              (31, 127, 160), (32, 500, 6016), (33, 40000, 64), (40, 20, 4096), (64, 193, 512), (65, 321, 288),
              (129, 700, 96)]
    for i, (M, N, K) in enumerate(shapes):
        for group in (32, 64, 128):
            t.check(M, N, K, group, (i + group // 32) % 2 == 0, ("bf16", "fp16")[i % 2], ("fp16", "bf16")[i // 2 % 2],
                    (i + group // 64) % 3 == 0, seed=i)
    assert gp.gemm_last_device_status() == 0
    print("all shapes right")
""")

FAULT = textwrap.dedent("""
    import sys, time
    sys.path.insert(0, {root!r})
    sys.path.insert(0, {tests!r})
    import torch
    import dense_gemm_preshuffle_gb300 as gp
    import test_gpu_w4g_tiles as t
    gp.load_library()
    _, W = t.weights({N}, {K}, 128, False, "bf16", 1)
    A = t.rows({M}, {K}, "bf16", 2)
    torch.cuda.synchronize()
    assert gp.gemm_last_device_status() == 0
    gp.gemm_debug_skip_load(2)
    t0 = time.time()
    gp.matmul_w4g(A, W, b_constant={b_constant!r})
    st = gp.gemm_last_device_status()
    assert st == 6, f"expected GP_ERR_DEVICE_TIMEOUT, got {{st}}"
    assert time.time() - t0 < 20
    t.check({M}, {N}, {K}, 128, False, "bf16", "bf16", False)
    assert gp.gemm_last_device_status() == 0
    print("next calls ok")
""")


def child(code, **env):
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, **env), capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


@pytest.mark.gpu
@pytest.mark.parametrize("tile", ["0", "1"])
def test_either_kernel_on_every_shape(tile):
    """A child process, because the choice is read once."""
    out = child(FORMS.format(root=ROOT, tests=os.path.dirname(__file__)), GP_W4G_TILE=tile)
    assert "all shapes right" in out


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,b_constant", [(40, 9000, 2048, False), (64, 21000, 1024, True), (32, 1500, 8192, False)])
def test_timeout_is_reported_and_the_context_survives(M, N, K, b_constant):
    """A stage's copies left out, as the bounded waits of the other kernels are tested."""
    out = child(FAULT.format(root=ROOT, tests=os.path.dirname(__file__), M=M, N=N, K=K, b_constant=b_constant),
                GP_W4G_TILE="1", GP_WAIT_LIMIT_MS="200")
    assert "next calls ok" in out
