"""Products with 4-bit group-scaled weights on the GPU: the packed layout byte
by byte, its inverse, and every element of every product against the 64-bit
definition and the error bounds of oracle.ffn."""
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


def f64(t):
    return t.double().cpu().numpy()


def make(N, K, group, zeros, scale_type, seed=0):
    """((codes, scales, zeros) as 64-bit-ready arrays, the packed weights)."""
    rng = np.random.default_rng(seed + 7 * N + K + group)
    groups = -(-K // group)
    codes = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    scales = torch.from_numpy((rng.random((N, groups)) + 0.5) / np.sqrt(K) / 4).to(TYPES[scale_type]).cuda()
    zp = rng.integers(0, 16, (N, groups), dtype=np.uint8) if zeros else None
    W = gp.preshuffle_w4g(torch.from_numpy(codes).cuda(), scales, group,
                          zeros=None if zp is None else torch.from_numpy(zp).cuda())
    return (codes, f64(scales), zp), W


def activations(M, K, dtype, seed=0, pad=8):
    rng = np.random.default_rng(seed + M + 3 * K)
    buf = torch.full((M, K + pad), float("nan"), dtype=TYPES[dtype], device="cuda")
    buf[:, :K] = torch.from_numpy(rng.standard_normal((M, K))).to(TYPES[dtype]).cuda()
    return buf[:, :K]


def within(got, want, bound):
    got = f64(got)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {want[bad][0]} +- {bound[bad][0]}")


@pytest.mark.parametrize("N,K,group,zeros", [(16, 128, 128, False), (33, 160, 32, True), (1, 32, 64, True),
                                             (7, 224, 128, True), (50, 320, 64, False)])
def test_packed_layout_and_round_trip(N, K, group, zeros):
    rng = np.random.default_rng(N + K)
    groups = -(-K // group)
    codes = torch.from_numpy(rng.integers(0, 256, (N, K // 2), dtype=np.uint8)).cuda()
    bits = rng.integers(0, 1 << 15, (N, groups), dtype=np.int16)
    scales = torch.from_numpy(bits).cuda().view(torch.bfloat16)
    zp = torch.from_numpy(rng.integers(0, 16, (N, groups), dtype=np.uint8)).cuda() if zeros else None
    W = gp.preshuffle_w4g(codes, scales, group, zeros=zp)
    want = ffn.w4g_pack(codes.cpu().numpy(), bits.view(np.uint16), None if zp is None else zp.cpu().numpy(), group)
    assert np.array_equal(W.packed.cpu().numpy(), want)
    c, s, z = gp.unpack_w4g(W)
    assert torch.equal(c, codes) and torch.equal(s.view(torch.int16), scales.view(torch.int16))
    assert (z is None) == (zp is None) and (z is None or torch.equal(z, zp))


SHAPES = [(1, 1, 32), (1, 16, 128), (1, 1000, 4096), (2, 17, 96), (3, 255, 160), (5, 64, 1056), (7, 300, 8320),
          (8, 128, 512), (9, 33, 2048), (15, 100, 64), (16, 512, 4096), (17, 65, 352), (24, 129, 256), (32, 96, 1024),
          (33, 70, 128), (65, 50, 288), (100, 40, 96)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype,scale_type,group,zeros", [
    ("bf16", "bf16", 128, False), ("fp16", "fp16", 32, True), ("bf16", "fp16", 64, True), ("fp16", "bf16", 128, False),
    ("bf16", "bf16", 32, True), ("fp16", "fp16", 64, False)])
def test_product(M, N, K, dtype, scale_type, group, zeros):
    w, W = make(N, K, group, zeros, scale_type)
    A = activations(M, K, dtype)
    buf = torch.full((M, N + 3), float("nan"), dtype=TYPES[dtype], device="cuda")
    out = gp.matmul_w4g(A, W, out=buf[:, :N])
    within(out, *ffn.w4g_bound(f64(A), [w], group, dtype))
    assert torch.isnan(buf[:, N:]).all()


@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 500, 1024), (2, 33, 160), (4, 16, 4096), (5, 300, 832), (8, 47, 96),
                                   (11, 130, 512), (16, 64, 2048), (20, 81, 288), (40, 30, 128)])
@pytest.mark.parametrize("dtype,act,group,zeros", [("bf16", "silu", 128, False), ("fp16", "gelu", 64, True),
                                                   ("bf16", "relu", 32, True)])
def test_gated_product(M, N, K, dtype, act, group, zeros):
    g, G = make(N, K, group, zeros, dtype, seed=1)
    u, U = make(N, K, group, zeros, dtype, seed=2)
    A = activations(M, K, dtype) * 4
    out = torch.full((M, N), float("nan"), dtype=TYPES[dtype], device="cuda")
    gp.matmul_w4g_gated(A, G, U, act=act, out=out)
    within(out, *ffn.w4g_bound(f64(A), [g, u], group, dtype, act))


@pytest.mark.parametrize("M,N,K", [(1, 500, 8192), (3, 1200, 4128), (12, 1100, 4256), (1, 2000, 2080), (8, 2400, 4096),
                                   (15, 1700, 2592), (40, 380, 5120)])
@pytest.mark.parametrize("dtype,group,zeros", [("bf16", 128, True), ("fp16", 32, False)])
def test_few_columns_and_long_sums(M, N, K, dtype, group, zeros):
    """Row tiles too few to fill the GPU: two or four blocks share each."""
    w, W = make(N, K, group, zeros, dtype, seed=10)
    u, U = make(N, K, group, zeros, dtype, seed=11)
    A = activations(M, K, dtype, seed=10)
    within(gp.matmul_w4g(A, W), *ffn.w4g_bound(f64(A), [w], group, dtype))
    first = gp.matmul_w4g_gated(A, W, U)
    within(first, *ffn.w4g_bound(f64(A), [w, u], group, dtype, "silu"))
    for _ in range(10):
        assert torch.equal(gp.matmul_w4g_gated(A, W, U, b_constant=True), first)


@pytest.mark.parametrize("M,N,K", [(16, 15000, 256), (20, 8000, 160), (8, 20000, 128)])
def test_many_columns(M, N, K):
    """Several units a block, in each of the forms that many row tiles take."""
    for group, dtype in ((128, "bf16"), (64, "fp16")):
        w, W = make(N, K, group, True, dtype, seed=12)
        A = activations(M, K, dtype, seed=12)
        within(gp.matmul_w4g(A, W), *ffn.w4g_bound(f64(A), [w], group, dtype))


def test_offset_codes_cancel():
    """A constant activation: the offset's share of the sum is thirty times the result."""
    N, K, group = 64, 2048, 128
    w, W = make(N, K, group, False, "bf16", seed=3)
    for dtype, value in (("bf16", 1.0), ("bf16", 3.0e4), ("fp16", 511.0), ("fp16", 2.0 ** -20)):
        A = torch.full((3, K), value, dtype=TYPES[dtype], device="cuda")
        C, bound = ffn.w4g_bound(f64(A), [w], group, dtype)
        within(gp.matmul_w4g(A, W), C, bound)


def test_extreme_codes_and_zero_points():
    N, K, group = 40, 256, 32
    A = activations(4, K, "fp16", seed=9)
    for code, zero in ((0, 15), (15, 0), (0, 0), (15, 15)):
        codes = torch.full((N, K // 2), code * 17, dtype=torch.uint8, device="cuda")
        scales = torch.full((N, K // group), 0.5, dtype=torch.float16, device="cuda")
        zp = torch.full((N, K // group), zero, dtype=torch.uint8, device="cuda")
        W = gp.preshuffle_w4g(codes, scales, group, zeros=zp)
        C, bound = ffn.w4g_bound(f64(A), [(codes.cpu().numpy(), f64(scales), zp.cpu().numpy())], group, "fp16")
        within(gp.matmul_w4g(A, W), C, bound)


@pytest.mark.parametrize("M", [1, 6])
def test_a_row_keeps_its_nan(M):
    w, W = make(70, 256, 64, False, "bf16", seed=4)
    A = activations(M + 2, 256, "bf16", seed=4)
    plain = gp.matmul_w4g(A, W)
    A[1] = 0
    A[2, 5] = float("nan")
    got = gp.matmul_w4g(A, W)
    assert not got[1].any() and torch.isnan(got[2]).all()
    keep = [i for i in range(M + 2) if i not in (1, 2)]
    assert torch.equal(got[keep], plain[keep])


@pytest.mark.parametrize("M,N,K", [(1, 300, 4096), (16, 100, 8192), (33, 64, 512)])
def test_repeats_are_bit_identical(M, N, K):
    _, W = make(N, K, 128, True, "bf16", seed=5)
    A = activations(M, K, "bf16", seed=5)
    first = gp.matmul_w4g(A, W)
    for _ in range(20):
        assert torch.equal(gp.matmul_w4g(A, W, b_constant=True), first)


def test_rows_do_not_depend_on_the_batch_around_them():
    """Row m of a batch is what it is alone, up to the order of fp32 sums."""
    w, W = make(96, 2048, 128, False, "bf16", seed=6)
    A = activations(32, 2048, "bf16", seed=6)
    for M in (1, 2, 8, 9, 16, 17, 31, 32):
        within(gp.matmul_w4g(A[:M], W), *ffn.w4g_bound(f64(A[:M]), [w], 128, "bf16"))


def test_chain_on_a_side_stream():
    _, W = make(512, 512, 64, True, "bf16", seed=7)
    A = activations(4, 512, "bf16", seed=7)
    want = A
    for _ in range(8):
        want = gp.matmul_w4g(want, W)
    torch.cuda.synchronize()
    side, got = torch.cuda.Stream(), A
    with torch.cuda.stream(side):
        for i in range(8):
            got = gp.matmul_w4g(got, W, b_constant=bool(i % 2))
    side.synchronize()
    assert torch.equal(got, want)


def test_empty_sizes():
    _, W = make(48, 64, 64, False, "bf16")
    z = dict(dtype=torch.bfloat16, device="cuda")
    assert gp.matmul_w4g(torch.empty((0, 64), **z), W).shape == (0, 48)
    E = gp.preshuffle_w4g(torch.empty((48, 0), dtype=torch.uint8, device="cuda"), torch.empty((48, 0), **z), 64)
    out = torch.full((3, 48), float("nan"), **z)
    gp.matmul_w4g(torch.empty((3, 0), **z), E, out=out)
    assert not torch.isnan(out).any() and not out.any()
    E = gp.preshuffle_w4g(torch.empty((0, 32), dtype=torch.uint8, device="cuda"), torch.empty((0, 1), **z), 64)
    assert gp.matmul_w4g(torch.zeros((3, 64), **z), E).shape == (3, 0)


def test_weights_past_32_bit_offsets():
    """Packed codes beyond 2^32 bytes: the last columns of a very wide matrix."""
    N, K, group = 1100000, 8192, 128
    gen = torch.Generator(device="cuda").manual_seed(2)
    codes = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.rand((N, K // group), generator=gen, device="cuda").div_(1000).to(torch.bfloat16)
    W = gp.preshuffle_w4g(codes, scales, group)
    A = activations(1, K, "bf16", seed=8)
    got = gp.matmul_w4g(A, W)
    for part in (slice(0, 64), slice(N - 64, N)):
        w = (codes[part].cpu().numpy(), f64(scales[part]), None)
        within(got[:, part], *ffn.w4g_bound(f64(A), [w], group, "bf16"))


def test_many_drawn_shapes():
    rng = np.random.default_rng(13)
    for i in range(30):
        M, N = (int(np.exp(rng.uniform(0, np.log(hi)))) for hi in (40, 900))
        K, group = 32 * int(rng.integers(1, 80)), (32, 64, 128)[i % 3]
        dtype = ("bf16", "fp16")[i % 2]
        w, W = make(N, K, group, i % 4 < 2, dtype, seed=30 + i)
        A = activations(M, K, dtype, seed=i)
        within(gp.matmul_w4g(A, W), *ffn.w4g_bound(f64(A), [w], group, dtype))


def test_refusals():
    z = dict(dtype=torch.bfloat16, device="cuda")
    w, W = make(32, 64, 64, False, "bf16")
    codes, scales = torch.zeros((32, 32), dtype=torch.uint8, device="cuda"), torch.zeros((32, 1), **z)
    for call in [
        lambda: gp.matmul_w4g(torch.zeros((2, 96), **z), W),
        lambda: gp.matmul_w4g(torch.zeros((2, 64), device="cuda"), W),
        lambda: gp.matmul_w4g(torch.zeros((64, 2), **z).t(), W),
        lambda: gp.matmul_w4g(torch.zeros((2, 64), **z), W, out=torch.zeros((2, 33), **z)),
        lambda: gp.preshuffle_w4g(codes, scales.float(), 64),
        lambda: gp.preshuffle_w4g(codes, scales, 32),
        lambda: gp.preshuffle_w4g(codes, scales, 0),
        lambda: gp.preshuffle_w4g(codes, scales, 64, zeros=scales),
        lambda: gp.matmul_w4g_gated(torch.zeros((2, 64), **z), W, W, act="exp"),
    ]:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(gp.GemmError) as e:
        gp.preshuffle_w4g(codes, torch.zeros((32, 4), **z), 16)
    assert e.value.code == 1
    with pytest.raises(gp.GemmError) as e:
        gp.preshuffle_w4g(torch.zeros((32, 24), dtype=torch.uint8, device="cuda"), torch.zeros((32, 1), **z), 64)
    assert e.value.code == 3
    with pytest.raises(gp.GemmError) as e:
        gp.matmul_w4g(torch.zeros((2, 68), **z)[:, :64], W)
    assert e.value.code == 3
