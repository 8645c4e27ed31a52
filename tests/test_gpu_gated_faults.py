"""The bounded waits of the gated products: a host-selected injection makes
the producers skip one stage load, the kernel's waits run out after a short
limit, it drains and exits, the host reads GP_ERR_DEVICE_TIMEOUT, and the next
calls on the same context are right.  In a child process, because the limit is
read once per process."""
import os
import subprocess
import sys
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = textwrap.dedent("""
    import sys, time
    sys.path.insert(0, {root!r})
    import torch
    import dense_gemm_preshuffle_gb300 as gp
    from oracle import ffn
    gp.load_library()
    gen = torch.Generator(device="cuda").manual_seed(3)
    t = lambda r, c, s=1.0: torch.randn((r, c), generator=gen, device="cuda").mul_(s).to(torch.bfloat16)
    M, N, K = 300, 520, 1024
    A, G, U, dH = t(M, K), t(N, K, 0.03), t(N, K, 0.03), t(M, N)
    forward = lambda: gp.gated_matmul(A, G, U, b_constant={b_constant!r})
    backward = lambda: gp.gated_matmul_backward(A, G, U, dH)
    calls = {{"forward": forward, "backward": backward}}
    torch.cuda.synchronize()
    assert gp.gemm_last_device_status() == 0
    gp.gemm_debug_skip_load(2)
    t0 = time.time()
    calls[{call!r}]()
    st = gp.gemm_last_device_status()
    assert st == 6, f"expected GP_ERR_DEVICE_TIMEOUT, got {{st}}"
    assert time.time() - t0 < 20
    f64 = lambda x: x.double().cpu().numpy()
    ops = [f64(x) for x in (A, G, U)]
    H, bound = ffn.gated_bound(*ops, "silu", "bf16")
    assert (abs(f64(forward()) - H) <= bound).all()
    want, bounds = ffn.gated_backward_bound(*ops, f64(dH), "silu", "bf16")
    for o, w, b in zip(backward(), want, bounds):
        assert (abs(f64(o) - w) <= b).all()
    assert gp.gemm_last_device_status() == 0
    print("next calls ok")
""")


@pytest.mark.gpu
@pytest.mark.parametrize("call,b_constant", [("forward", False), ("forward", True), ("backward", False)])
def test_timeout_is_reported_and_the_context_survives(call, b_constant):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dense_gemm_preshuffle_gb300 import build
    build.build()
    env = dict(os.environ, GP_WAIT_LIMIT_MS="200")
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT, call=call, b_constant=b_constant)], env=env,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "next calls ok" in r.stdout
