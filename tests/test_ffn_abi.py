"""Host-side argument checks of the feed-forward entry points, their packed
sizes and the binding's refusals (no GPU: every call returns before the
device is touched)."""
import ctypes

import numpy as np
import pytest
import torch

import dense_gemm_preshuffle_gb300 as gp
from dense_gemm_preshuffle_gb300 import build
from oracle import ffn

FAKE = 0x10000  # an aligned, never-dereferenced address


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gp.load_library()


RUN = dict(A=FAKE, lda=512, G=FAKE, ldg=512, U=FAKE, ldu=512, dtype=0, M=16, N=256, K=512, act=2, H=FAKE, ldh=256,
           flags=0)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=99), 1), (dict(dtype=-1), 1), (dict(dtype=1), 2), (dict(dtype=6), 2),
    (dict(act=0), 1), (dict(act=4), 1), (dict(flags=4), 1),
    (dict(M=-1), 3), (dict(N=-1), 3), (dict(K=-1), 3), (dict(M=1 << 31), 3), (dict(K=1 << 31), 3),
    (dict(lda=504), 3), (dict(ldg=513), 3), (dict(ldu=520, K=521), 3), (dict(ldh=248), 3), (dict(ldh=257, N=257), 3),
    (dict(lda=1 << 38), 3),
    (dict(A=None), 1), (dict(G=None), 1), (dict(U=None), 1), (dict(H=None), 1),
    (dict(A=FAKE + 8), 4), (dict(G=FAKE + 2), 4), (dict(U=FAKE + 4), 4), (dict(H=FAKE + 8), 4),
    (dict(M=0, A=None, H=None), 0), (dict(N=0, G=None, U=None, H=None), 0),
])
def test_gated_run_checks(lib, change, code):
    a = {**RUN, **change}
    assert lib.gemm_gated_run(*[a[k] for k in RUN], None) == code


BACK = dict(A=FAKE, lda=512, G=FAKE, ldg=512, U=FAKE, ldu=512, dH=FAKE, lddh=256, dtype=5, M=16, N=256, K=512, act=3,
            dA=FAKE, ldda=512, dG=FAKE, lddg=512, dU=FAKE, lddu=512, ws=FAKE, wsb=1 << 40)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=7), 2), (dict(dtype=8), 1), (dict(act=0), 1), (dict(M=-1), 3), (dict(N=1 << 31), 3),
    (dict(lddh=255), 3), (dict(ldda=511), 3), (dict(lddg=8), 3), (dict(lddu=516), 3),
    (dict(dG=None), 1), (dict(dU=None), 1), (dict(dH=None), 1), (dict(ws=None), 1), (dict(wsb=15), 3),
    (dict(dA=FAKE + 8), 4), (dict(dG=FAKE + 8), 4), (dict(dU=FAKE + 8), 4), (dict(dH=FAKE + 8), 4),
    (dict(ws=FAKE + 8), 4),
    (dict(dA=None, dG=None, dU=None), 0), (dict(M=0, N=0), 0), (dict(K=0), 0),
    # the pitches of outputs that are not wanted are not looked at
    (dict(dA=None, ldda=1, M=0, N=0), 0),
])
def test_gated_backward_checks(lib, change, code):
    a = {**BACK, **change}
    assert lib.gemm_gated_backward(*[a[k] for k in BACK], None) == code


def test_gated_workspace(lib):
    for M, N, K in ((1, 1, 1), (128, 1024, 512), (8192, 8192, 4096)):
        # room for dg and du at least
        assert gp.gemm_gated_backward_workspace_bytes(M, N, K) >= 4 * M * N
    for dims in ((0, 5, 5), (5, 0, 5), (5, 5, 0)):
        assert gp.gemm_gated_backward_workspace_bytes(*dims) == 0
    with pytest.raises(gp.GemmError) as e:
        gp.gemm_gated_backward_workspace_bytes(-1, 2, 2)
    assert e.value.code == 3
    assert lib.gemm_gated_backward_workspace_bytes(1, 1, 1, None) == 1


@pytest.mark.parametrize("N,K,group,zeros", [(16, 128, 128, 0), (17, 128, 32, 1), (1, 32, 64, 1), (100, 8320, 64, 0)])
def test_w4g_sizes(lib, N, K, group, zeros):
    rng = np.random.default_rng(3)
    groups = -(-K // group)
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    sc = rng.integers(0, 1 << 16, (N, groups), dtype=np.uint16)
    zp = rng.integers(0, 16, (N, groups), dtype=np.uint8) if zeros else None
    assert gp.gemm_packed_w4g_bytes(N, K, group, zeros) == ffn.w4g_pack(codes, sc, zp, group).size


@pytest.mark.parametrize("N,K,group,zeros,code", [
    (16, 128, 16, 0, 1), (16, 128, 0, 0, 1), (16, 128, 128, 2, 1), (16, 130, 128, 0, 3), (-1, 128, 128, 0, 3),
    (16, -32, 32, 0, 3), (1 << 31, 128, 128, 0, 3), (0, 0, 32, 1, 0),
])
def test_w4g_shape_rules(lib, N, K, group, zeros, code):
    out = ctypes.c_size_t(7)
    assert lib.gemm_packed_w4g_bytes(N, K, group, zeros, ctypes.byref(out)) == code
    assert lib.gemm_packed_w4g_bytes(N, K, group, zeros, None) == 1
    if zeros < 2:
        z = FAKE if zeros else None
        assert lib.gemm_preshuffle_w4g(FAKE, FAKE, z, N, K, group, FAKE, None) == code if code else True
        assert lib.gemm_unpack_w4g(FAKE, N, K, group, zeros, FAKE, FAKE, z, None) == code if code else True


@pytest.mark.parametrize("which", ["codes", "scales", "packed"])
def test_w4g_pack_pointers(lib, which):
    a = dict(codes=FAKE, scales=FAKE, zeros=None, N=16, K=128, group=64, packed=FAKE)
    assert lib.gemm_preshuffle_w4g(*{**a, which: None}.values(), None) == 1
    assert lib.gemm_preshuffle_w4g(*{**a, which: FAKE + 4}.values(), None) == 4
    # zero points go out where, and only where, they were packed
    assert lib.gemm_unpack_w4g(FAKE, 16, 128, 64, 1, FAKE, FAKE, None, None) == 1
    assert lib.gemm_unpack_w4g(FAKE, 16, 128, 64, 0, FAKE, FAKE, FAKE, None) == 1


W4 = dict(A=FAKE, lda=512, dtype=0, W=FAKE, U=None, sd=0, zeros=0, M=3, N=100, K=512, group=128, act=0, C=FAKE,
          ldc=100, flags=0)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=2), 2), (dict(dtype=50), 1), (dict(sd=6), 2), (dict(sd=-3), 1), (dict(zeros=5), 1),
    (dict(group=48), 1), (dict(K=100), 3), (dict(lda=511), 3), (dict(lda=504), 3), (dict(ldc=99), 3), (dict(M=-2), 3),
    (dict(M=1 << 31), 3), (dict(act=1), 1), (dict(U=FAKE), 1), (dict(U=FAKE, act=4), 1), (dict(flags=8), 1),
    (dict(A=None), 1), (dict(W=None), 1), (dict(C=None), 1), (dict(A=FAKE + 8), 4), (dict(W=FAKE + 8), 4),
    (dict(U=FAKE + 8, act=1), 4), (dict(C=FAKE + 2), 4), (dict(M=0, A=None, C=None), 0), (dict(N=0, C=None), 0),
])
def test_w4g_run_checks(lib, change, code):
    a = {**W4, **change}
    assert lib.gemm_run_w4g(*[a[k] for k in W4], None) == code


def test_binding_refuses_on_the_host():
    a = torch.zeros((4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # CPU tensors
        gp.gated_matmul(a, a, a)
    with pytest.raises(ValueError):
        gp.gated_matmul(a.float(), a, a)
    with pytest.raises(ValueError):
        gp.preshuffle_w4g(torch.zeros((4, 64), dtype=torch.uint8), a, 128)
    w = gp.W4Weights(a, 4, 64, 32, 0, False)
    with pytest.raises(ValueError):
        gp.matmul_w4g(a, w)
    with pytest.raises(ValueError):  # the two halves differ
        gp.matmul_w4g_gated(a, w, w._replace(group=64))


# ------------------------------------------------------------ the definitions themselves

@pytest.mark.parametrize("name", ["relu", "silu", "gelu"])
def test_slopes_against_differences(name):
    v = np.linspace(-9.0, 9.0, 1800)  # 0 is not among them
    h = 1e-6
    d = (ffn.act(v + h, name) - ffn.act(v - h, name)) / (2 * h)
    assert np.max(np.abs(d - ffn.act_slope(v, name))) < 1e-8


@pytest.mark.parametrize("name", ["relu", "silu", "gelu"])
def test_gradients_against_differences(name):
    rng = np.random.default_rng(5)
    M, N, K = 5, 7, 6
    A, G, U = rng.standard_normal((M, K)), rng.standard_normal((N, K)), rng.standard_normal((N, K))
    dH = rng.standard_normal((M, N))
    grads = ffn.gated_backward(A, G, U, dH, name)
    h = 1e-5
    for i in range(3):
        v = rng.standard_normal((A, G, U)[i].shape)
        up = [x + h * v if j == i else x for j, x in enumerate((A, G, U))]
        dn = [x - h * v if j == i else x for j, x in enumerate((A, G, U))]
        num = ((ffn.gated(*up, name) - ffn.gated(*dn, name)) * dH).sum() / (2 * h)
        assert abs(num - (grads[i] * v).sum()) < 1e-6 * (1 + abs(num))


def test_dequantize_by_hand():
    codes = np.array([[0x21, 0x43]], dtype=np.uint8).repeat(16, axis=1)  # K = 64
    scales, zeros = np.array([[0.5, 2.0]]), np.array([[1, 3]], dtype=np.uint8)
    w = ffn.w4g_dequantize(codes, scales, zeros, 32)
    assert w[0, 0] == 0.0 and w[0, 1] == 0.5          # (1 - 1) / 2, (2 - 1) / 2
    assert w[0, 62] == 0.0 and w[0, 63] == 2.0        # (3 - 3) * 2, (4 - 3) * 2
    assert ffn.w4g_dequantize(codes, scales, None, 32)[0, 63] == -8.0


def test_sizes_past_any_memory(lib):
    big = (1 << 31) - 1
    out = ctypes.c_size_t(0)
    assert lib.gemm_gated_backward_workspace_bytes(big, big, 8, ctypes.byref(out)) == 3
    assert lib.gemm_packed_w4g_bytes(big, big - 31, 128, 0, ctypes.byref(out)) == 3
    a = {**RUN, "M": big, "N": big, "ldh": 1 << 31}
    assert lib.gemm_gated_run(*[a[k] for k in RUN], None) == 3
    assert gp.gemm_gated_backward_workspace_bytes(1 << 20, 1 << 20, 64) >= 4 << 40
