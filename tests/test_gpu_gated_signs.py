"""ReLU's gradients where a gate is within rounding of 0.  The slope jumps
there, so a sum whose sign comes out wrong adds or loses a whole term."""
import numpy as np
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


@pytest.mark.parametrize("M,N,K", [(1100, 1500, 1000), (600, 5000, 2051)])
def test_gates_within_rounding_of_zero(M, N, K):
    """Gates of 1e-8 among sums of size 1, one to a 32 x 32 block: each made by
    choosing the weight beside one large, one small and one tiny activation."""
    rng = np.random.default_rng(M)
    A = rng.standard_normal((M, K)).astype(np.float16)
    G, U = ((rng.standard_normal((N, K)) / np.sqrt(K)).astype(np.float16) for _ in range(2))
    dH = rng.standard_normal((M, N)).astype(np.float16)
    A[:, 0], A[:, 1], A[:, 2] = 1.0, 2.0 ** -6, 2.0 ** -12
    pairs = [(32 * (i % (M // 32)) + 5 * i % 32, 32 * i + 7 * i % 32) for i in range(N // 32)]
    for m, n in pairs:
        dH[m, n] = 2.0
        for k in (0, 1, 2):  # each leaves the rounding of its weight times its activation
            G[n, k] = 0
            rest = A[m].astype(np.float64) @ G[n].astype(np.float64)
            G[n, k] = np.clip(-rest / float(A[m, k]), -64, 64)
    a, g, u, d = (x.astype(np.float64) for x in (A, G, U, dH))
    gate, up = a @ g.T, a @ u.T
    at = np.array(pairs)
    tiny = gate[at[:, 0], at[:, 1]]
    assert (np.abs(tiny) < 1e-5).all() and (np.abs(tiny) < 2e-7).sum() > len(pairs) // 4
    assert (tiny > 0).any() and (tiny < 0).any()
    dG = (d * up * (gate > 0)).T @ a

    def padded(x):
        buf = torch.zeros((x.shape[0], (x.shape[1] + 7) // 8 * 8), dtype=torch.float16, device="cuda")
        buf[:, :x.shape[1]] = torch.from_numpy(x).cuda()
        return buf[:, :x.shape[1]]

    got = gp.gated_matmul_backward(*(padded(x) for x in (A, G, U, dH)), act="relu")[1].double().cpu().numpy()
    off = got - dG
    for m, n in pairs:
        # the term that a wrong sign adds or loses is 2 u A[m]; the roundings'
        # share along A[m] is a thousandth of a gradient's size, under 0.1
        term = 2.0 * up[m, n]
        if gate[m, n] == 0.0 or abs(term) < 0.4:
            continue
        along = off[n] @ a[m] / (a[m] @ a[m])
        assert abs(along) < 0.5 * abs(term), (m, n, gate[m, n], along, term)
