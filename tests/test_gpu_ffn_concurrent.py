"""Every kernel of the gated products and of the 4-bit weights launched
together on four streams, six rounds: each output has the bits of the same
call run alone."""
import pytest
import torch

import dense_gemm_preshuffle_gb300 as gp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_gemm_preshuffle_gb300 import build
    build.build()
    gp.load_library()


def test_four_streams():
    gen = torch.Generator(device="cuda").manual_seed(12)

    def rows(r, c, scale=1.0):
        return torch.randn((r, c), generator=gen, device="cuda").mul_(scale).to(torch.bfloat16)

    def packed(N, K, group):
        codes = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
        scales = torch.rand((N, K // group), generator=gen, device="cuda").div_(K ** 0.5).to(torch.bfloat16)
        return gp.preshuffle_w4g(codes, scales, group)

    calls = []
    # the streaming kernel alone and in clusters; weights as rows alone, in
    # clusters and in several units; tiles of pairs
    for M, N, K in ((1, 3000, 1024), (2, 300, 4096), (64, 4096, 512), (64, 500, 4096), (200, 9000, 256), (700, 1500, 704)):
        A, G, U = rows(M, K), rows(N, K, K ** -0.5), rows(N, K, K ** -0.5)
        calls.append(lambda A=A, G=G, U=U: (gp.gated_matmul(A, G, U),))
    # gradients in parts and whole
    for M, N, K in ((300, 504, 2048), (40, 1200, 704), (600, 1400, 640)):
        A, G, U, dH = rows(M, K), rows(N, K, K ** -0.5), rows(N, K, K ** -0.5), rows(M, N)
        calls.append(lambda A=A, G=G, U=U, dH=dH: gp.gated_matmul_backward(A, G, U, dH, act="relu"))
    # 4-bit weights: streaming alone and in clusters, tiles alone and in clusters
    for M, N, K in ((3, 6000, 1024), (1, 300, 4096), (40, 20000, 512), (33, 1500, 4096)):
        A, W, V = rows(M, K), packed(N, K, 128), packed(N, K, 128)
        calls.append(lambda A=A, W=W: (gp.matmul_w4g(A, W),))
        calls.append(lambda A=A, W=W, V=V: (gp.matmul_w4g_gated(A, W, V),))
    alone = [call() for call in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for turn in range(6):
        got = []
        for i, call in enumerate(calls):
            with torch.cuda.stream(streams[(i + turn) % 4]):
                got.append(call())
        torch.cuda.synchronize()
        for i, (want, have) in enumerate(zip(alone, got)):
            assert all(torch.equal(w, h) for w, h in zip(want, have)), (turn, i)
    assert gp.gemm_last_device_status() == 0
