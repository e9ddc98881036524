"""The cross entropy of rows whose target is nearly certain: the loss is not a difference of two large numbers.

With S the sum over the other entries of exp(z_v - z_y), the loss is log(1 + S).  Bars: a logit is off by at most bz (as in
test_gpu_cross_entropy), which moves S by a factor of at most exp(2 bz); an exponential is within 2^-20 of its value, its
argument |d| within 2^-22 |d| (d <= 100 wherever the term counts: 2^-15); and every addition to a sum of 1 or more is off by
at most half a step, 2^-24 of it up to 2, but never by more than what is added: N additions by min(S, N 2^-24).  At the
end one addition and a logarithm: 2^-22 of the loss.
"""
import math

import pytest

from tests import test_gpu_cross_entropy as C

pytestmark = pytest.mark.gpu
mx = C.mx


def confident(T, H, V, margin, seed):
    """Rows along their target's weights: z_y = margin, the others about margin / sqrt(H)."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randn((V, H), generator=gen, device="cuda").bfloat16()
    y = torch.randint(0, V, (T,), generator=gen, device="cuda")
    wt = w[y].float()
    x = (margin * (0.9 + 0.1 * torch.rand((T, 1), generator=gen, device="cuda")) * wt /
         (wt * wt).sum(-1, keepdim=True)).bfloat16()
    return x, w, y


@pytest.mark.parametrize("T,H,V", [(1, 512, 1000), (20, 512, 1000), (32, 1024, 300), (50, 512, 1000), (300, 512, 3000),
                                   (1000, 1024, 4000)])
@pytest.mark.parametrize("margin", [12.0, 40.0, 150.0, 900.0])
def test_losses_of_nearly_certain_targets(mx, T, H, V, margin):
    import torch
    x, w, y = confident(T, H, V, margin, seed=T + V)
    loss, lse = mx.linear_cross_entropy_fwd(x, w, y)
    C.check_forward(loss, lse, x, w, y)
    assert (loss >= 0).all()
    z, bz = C.bars_of_logits(x, w)
    d = z - z.gather(1, y[:, None])
    d.scatter_(1, y[:, None], -math.inf)
    assert (d < 0).all()                      # the target is the largest
    S = torch.exp(d).sum(1)
    want = torch.log1p(S)
    bz = bz.amax(1)
    adds = 128 + 40 + V / 128
    bar = S * (torch.expm1(2 * bz) + 2.0 ** -20 + 2.0 ** -15) + torch.minimum(S, torch.full_like(S, adds * 2.0 ** -24))
    bar = bar * 1.01 + 2.0 ** -22 * want + 1e-38
    err = (loss.double() - want).abs()
    assert (err <= bar).all(), float((err / bar).max())


@pytest.mark.parametrize("T", [7, 100, 3000])
def test_no_loss_is_negative(mx, T):
    """The likeliest entry as every row's target, from flat rows to peaked ones."""
    import torch
    for scale in (0.5, 5.0, 50.0, 500.0):
        x, w, _ = C.make(T, 256, 500, seed=3, ignored=0.0, lean=0.0, scale=scale)
        y = (x.double() @ w.double().t()).argmax(1)
        loss, _ = mx.linear_cross_entropy_fwd(x, w, y)
        assert (loss >= 0).all()


@pytest.mark.parametrize("T,H,V", [(1, 2048, 1000), (20, 4096, 1000), (32, 2048, 300), (50, 4096, 3000), (64, 2048, 300),
                                   (300, 2048, 3000), (1000, 4096, 2000), (1100, 4096, 2000), (3000, 2048, 4000)])
@pytest.mark.parametrize("margin", [50.0, 150.0, 900.0])
def test_gradients_of_nearly_certain_targets(mx, T, H, V, margin):
    """S is below 2^-40 here: lse is the target's logit to the bit, and the backward's logits are the forward's, so p is 1
    and dz 0 at the target; at the others dz is p, in all S: dx is within S max|w| of 0 (S moved by exp(2 bz) and the
    roundings of 2^-8), dw within the sum of S |x| over the rows."""
    import torch
    x, w, y = confident(T, H, V, margin, seed=T + V)
    _, lse = mx.linear_cross_entropy_fwd(x, w, y)
    z, bz = C.bars_of_logits(x, w)
    d = z - z.gather(1, y[:, None])
    d.scatter_(1, y[:, None], -math.inf)
    S = torch.exp(d + 2 * bz.amax(1)[:, None]).sum(1)
    assert S.max() < 2.0 ** -40
    dx, dw = mx.linear_cross_entropy_bwd(torch.ones(T, device="cuda"), x, w, y, lse)
    assert (dx.double().abs() <= 1.1 * S[:, None] * w.double().abs().max() + 1e-38).all()
    assert (dw.double().abs() <= 1.1 * (S[:, None] * x.double().abs()).sum(0) + 1e-38).all()
