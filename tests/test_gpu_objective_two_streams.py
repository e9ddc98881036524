"""Two calls in flight at once, each on a stream and with a workspace of its own: few rows beside a training batch, and the
router beside both.  Every wait of these kernels is for CTAs that run already, whatever else holds the SMs; results are those
of the calls one after the other."""
import pytest

from tests import test_gpu_cross_entropy as C

pytestmark = pytest.mark.gpu
mx = C.mx


@pytest.mark.parametrize("sizes", [((20, 512, 9000), (1500, 512, 9000)), ((60, 1024, 20000), (50, 1024, 20000)),
                                   ((300, 256, 4000), (1200, 256, 60000)), ((2000, 256, 4000), (2000, 128, 5000))])
def test_two_cross_entropies_and_a_router_at_once(mx, sizes):
    import torch
    work = []
    for T, H, V in sizes:
        x, w, y = C.make(T, H, V, seed=T)
        logits = torch.randn((20 * T, 64), device="cuda")
        ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in
              (mx.linear_cross_entropy_workspace_size(T, H, V), mx.linear_cross_entropy_bwd_workspace_size(T, H, V),
               max(16, mx.moe_route_workspace_size(20 * T, 64, 4)))]
        work.append((x, w, y, logits, torch.rand(T, device="cuda"), ws))

    def step(x, w, y, logits, dloss, ws):
        loss, lse = mx.linear_cross_entropy_fwd(x, w, y, workspace=ws[0])
        routed = mx.moe_route_fwd(logits, 4, workspace=ws[2])
        return loss, lse, *routed, *mx.linear_cross_entropy_bwd(dloss, x, w, y, lse, workspace=ws[1])
    want = [step(*a) for a in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    got = [None] * len(work)
    for _ in range(30):
        for i, (s, a) in enumerate(zip(streams, work)):
            with torch.cuda.stream(s):
                got[i] = step(*a)
    torch.cuda.synchronize()
    for a, b, g in zip(work, want, got):
        assert all(torch.equal(p, q) for p, q in zip(b, g))
        assert mx.mxfp8_check_device_error(a[5][0]) == (0, 0) and mx.mxfp8_check_device_error(a[5][1]) == (0, 0)
