"""The operators together, as examples/feed_forward.py uses them: the loss of
the trained block falls, and the block with 4-bit weights stays near it.  And
both forms of the gated products, streaming and tensor-core tiles, forced on
every shape in child processes (the switch is read once per process)."""
import importlib.util
import os
import subprocess
import sys
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_gemm_preshuffle_gb300 import build
    build.build()


@pytest.mark.gpu
def test_example_trains_and_serves():
    import dense_gemm_preshuffle_gb300 as gp
    gp.load_library()
    spec = importlib.util.spec_from_file_location("feed_forward", os.path.join(ROOT, "examples", "feed_forward.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, off = example.run(tokens=512, width=256, hidden=640, steps=12)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
    # 4 bits a weight: the rounding error of a weight is uniform within half of
    # a fifteenth of its group's range, about 6 standard deviations of normal
    # weights: 0.12 of a weight's deviation each, in three matrices
    assert 0.0 < off < 3 * 0.12
    assert gp.gemm_last_device_status() == 0


FORMS = textwrap.dedent("""
    import sys
    sys.path.insert(0, {root!r})
    import torch
    import dense_gemm_preshuffle_gb300 as gp
    from oracle import ffn
    gp.load_library()
    gen = torch.Generator(device="cuda").manual_seed(4)
    t = lambda r, c, s=1.0: torch.randn((r, (c + 7) // 8 * 8), generator=gen, device="cuda").mul_(s).to(torch.float16)[:, :c]
    f64 = lambda x: x.double().cpu().numpy()
    for M, N, K in ((1, 100, 72), (3, 513, 640), (9, 64, 1000), (17, 250, 129), (40, 700, 64), (64, 128, 128),
                    (65, 129, 257), (200, 300, 320), (257, 40, 90), (500, 260, 65)):
        A, G, U, dH = t(M, K), t(N, K, K ** -0.5), t(N, K, K ** -0.5), t(M, N)
        ops = [f64(x) for x in (A, G, U)]
        H, bound = ffn.gated_bound(*ops, "gelu", "fp16")
        assert (abs(f64(gp.gated_matmul(A, G, U, act="gelu")) - H) <= bound).all(), (M, N, K)
        want, bounds = ffn.gated_backward_bound(*ops, f64(dH), "gelu", "fp16")
        for o, w, b in zip(gp.gated_matmul_backward(A, G, U, dH, act="gelu"), want, bounds):
            assert (abs(f64(o) - w) <= b).all(), (M, N, K)
    assert gp.gemm_last_device_status() == 0
    print("all shapes right")
""")


@pytest.mark.gpu
@pytest.mark.parametrize("stream", ["0", "1"])
def test_either_form_on_every_shape(stream):
    r = subprocess.run([sys.executable, "-c", FORMS.format(root=ROOT)], env=dict(os.environ, GP_GATED_STREAM=stream),
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "all shapes right" in r.stdout
