"""The first call of a process inside a graph capture: what a call prepares once per device must not need the stream."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def _child():
    import torch

    import mxfp8_block_scaled_03_gb300 as mx
    mx.lib()
    T, H, V, E, k = 200, 64, 3000, 16, 2
    x = torch.randn(T, H, device="cuda").bfloat16()
    w = (0.1 * torch.randn(V, H, device="cuda")).bfloat16()
    y = torch.randint(0, V, (T,), device="cuda")
    logits, dloss = torch.randn(2000, E, device="cuda"), torch.ones(T, device="cuda")
    torch.cuda.synchronize()

    def step():
        loss, lse = mx.linear_cross_entropy_fwd(x, w, y)
        routed = mx.moe_route_fwd(logits, k)
        return (loss, lse, *mx.linear_cross_entropy_bwd(dloss, x, w, y, lse), *routed,
                mx.moe_route_bwd(logits, *routed[:4], dgates=torch.ones_like(routed[1])),
                *mx.linear_cross_entropy_fwd(x[:5], w, y[:5]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(captured, step()))
    print("captured ok", flush=True)


def test_first_call_inside_a_capture():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from mxfp8_block_scaled_03_gb300 import build_ext
    build_ext.build()
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured ok" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]


if __name__ == "__main__":
    _child()
