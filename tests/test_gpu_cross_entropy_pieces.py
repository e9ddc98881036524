"""linear_cross_entropy_bwd where dz is half of the logits at a time: several pieces of the vocabulary, their dx added up in
one or several shares, within exactly the workspace that is asked for.  Bars as in test_gpu_cross_entropy; every further
piece is one more fp32 addition, which its (V / 16 + 40) terms cover."""
import pytest

from tests import test_gpu_cross_entropy as C

pytestmark = pytest.mark.gpu
mx = C.mx


# packed rows in several shares or one, with hardly a row left, a last piece of few entries; rows as they are; more than
# 65536 rows, whose pieces are the smallest
@pytest.mark.parametrize("T,H,V,ignored", [(600, 64, 120000, 0.3), (1000, 72, 100001, 0.0), (2048, 4096, 17000, 0.1),
                                           (1100, 264, 60000, 0.3), (1500, 520, 50257, 0.9), (2000, 136, 40000, 0.999),
                                           (1024, 128, 131329, 0.2), (500, 64, 200000, 0.3), (300, 72, 270001, 0.0),
                                           (66000, 16, 4100, 0.5), (3000, 1024, 30001, 0.0)])
def test_pieces(mx, T, H, V, ignored):
    import torch
    x, w, y = C.make(T, H, V, seed=T + V, ignored=ignored)
    y[0] = V - 1
    loss, lse = mx.linear_cross_entropy_fwd(x, w, y)
    gen = torch.Generator(device="cuda").manual_seed(1)
    dloss = torch.rand(T, generator=gen, device="cuda") / T
    dlse = 0.1 * torch.randn(T, generator=gen, device="cuda") / T
    n = mx.linear_cross_entropy_bwd_workspace_size(T, H, V)
    buf = torch.full((n + 4096,), 255, dtype=torch.uint8, device="cuda")
    out = torch.full_like(x, 7.0), torch.full_like(w, 7.0)
    dx, dw = mx.linear_cross_entropy_bwd(dloss, x, w, y, lse, dlse=dlse, out=out, workspace=buf[:n])
    assert mx.mxfp8_check_device_error(buf) == (0, 0)
    assert (buf[n:] == 255).all()
    C.check_backward(dx, dw, dloss, dlse, x, w, y, lse)
    again = mx.linear_cross_entropy_bwd(dloss, x, w, y, lse, dlse=dlse)
    assert all(torch.equal(a, b) for a, b in zip((dx, dw), again))


@pytest.mark.parametrize("T,H,V", [(600, 64, 120000), (500, 64, 200000), (2048, 4096, 17000), (1100, 264, 60000)])
def test_rows_without_a_target_hold_anything(mx, T, H, V):
    import torch
    x, w, y = C.make(T, H, V, seed=5)
    _, lse = mx.linear_cross_entropy_fwd(x, w, y)
    dloss = torch.rand(T, device="cuda") / T
    clean = mx.linear_cross_entropy_bwd(dloss, x, w, y, lse)
    off = y < 0
    for t, v in ((x, float("nan")), (lse, float("inf")), (dloss, float("nan"))):
        t[off] = v
    dirty = mx.linear_cross_entropy_bwd(dloss, x, w, y, lse)
    assert all(torch.equal(a, b) for a, b in zip(clean, dirty)) and not dirty[0][off].any()
