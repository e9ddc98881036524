"""Failure detection of the cross entropy's kernels on the GPU without a fault: a pipeline wait that runs out sets a bit
of the error word, every role drains and exits, and the next call on the same workspace is as good as the first.

MXFP8MOE_WAIT_LIMIT_NS = 1000 makes the waits run out: the accumulator of a tile takes several microseconds.  Run in a
child process, so that no other test sees the variable.
"""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def _child(T, H, V):
    import torch

    import mxfp8_block_scaled_03_gb300 as mx
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((T, H), generator=gen, device="cuda").bfloat16()
    w = (0.02 * torch.randn((V, H), generator=gen, device="cuda")).bfloat16()
    y = torch.randint(0, V, (T,), generator=gen, device="cuda")
    dloss = torch.ones(T, device="cuda")
    wf = torch.empty(mx.linear_cross_entropy_workspace_size(T, H, V), dtype=torch.uint8, device="cuda")
    wb = torch.empty(mx.linear_cross_entropy_bwd_workspace_size(T, H, V), dtype=torch.uint8, device="cuda")

    def both(lse=None):
        loss, got = mx.linear_cross_entropy_fwd(x, w, y, workspace=wf)
        f = mx.mxfp8_check_device_error(wf)
        grads = mx.linear_cross_entropy_bwd(dloss, x, w, y, got if lse is None else lse, workspace=wb)
        return (loss, got, *grads), f, mx.mxfp8_check_device_error(wb)
    first, f, b = both()
    assert f == (0, 0) and b == (0, 0), (f, b)
    os.environ["MXFP8MOE_WAIT_LIMIT_NS"] = "1000"
    try:
        _, f, b = both(first[1])
    finally:
        os.environ.pop("MXFP8MOE_WAIT_LIMIT_NS")
    for st, bits in (f, b):
        assert st == mx.ERR_DEVICE_TIMEOUT and bits & 0x1F00, (st, hex(bits))
    again, f, b = both()
    assert f == (0, 0) and b == (0, 0), (f, b)
    assert all(torch.equal(p, q) for p, q in zip(first, again))
    print("timeout path ok", flush=True)


@pytest.mark.parametrize("T,H,V", [(40, 16384, 20000), (100, 16384, 3000), (1500, 16384, 4000)],
                         ids=["few_rows", "single_cta", "cta_pairs"])
def test_waits_that_run_out_are_reported(T, H, V):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from mxfp8_block_scaled_03_gb300 import build_ext
    build_ext.build()
    env = dict(os.environ)
    env.pop("MXFP8MOE_WAIT_LIMIT_NS", None)
    r = subprocess.run([sys.executable, os.path.abspath(__file__), str(T), str(H), str(V)], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "timeout path ok" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]


if __name__ == "__main__":
    _child(*map(int, sys.argv[1:]))
