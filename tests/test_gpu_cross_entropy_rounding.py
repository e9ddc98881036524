"""What the cross entropy's gradient does beyond rounding dz to bf16: two pieces of it up to 64 rows, and dz relative to
the largest weight.  Each bar is shown to notice its loss, on a model of the gradient with that loss planted in it.

Two pieces.  Let e be the error of a result before its own rounding, `want` the exact value: rounding both to bf16 gives
equal numbers but with probability |e| / step, when they are a step of at most 2^-7 |want| apart.  So the norm of their
difference is at most sqrt(2^-7 delta) of want's, with delta the norm of e relative to want's.  dz is off by 2^-16 of its
value, its logit by bz (see test_gpu_cross_entropy) and its exponential by 2^-20 + 2^-21 (|z| + |lse|), errors of their own in
every entry, so delta is at most their sum.

Weights.  Where every row has the weight s = (1 + 2^-8) / 1024 and p is below 2^-10, dz / s is p - 1 at the target, and
rounding it is off by at most 2^-10; s itself rounded to bf16 loses its 2^-8 in every row, and so in the coefficient of
the result on the exact one.  Independent roundings of 2^-8 leave 2^-8 / sqrt(T) of that.
"""
import math

import pytest

from tests import test_gpu_cross_entropy as C

pytestmark = pytest.mark.gpu
mx = C.mx


def exact_dz(x, w, y, lse, dloss):
    import torch
    z = x.double() @ w.double().t()
    dz = dloss.double()[:, None] * torch.exp(z - lse.double()[:, None])
    dz.scatter_add_(1, y.long()[:, None], -dloss.double()[:, None])
    return z, dz


@pytest.mark.parametrize("T", [5, 16, 20, 32, 50, 64])
def test_up_to_64_rows_dz_has_two_pieces(mx, T):
    import torch
    H, V = 64, 3000
    x, w, y = C.make(T, H, V, seed=T, ignored=0.0)
    _, lse = mx.linear_cross_entropy_fwd(x, w, y)
    gen = torch.Generator(device="cuda").manual_seed(T)
    dloss = 0.5 + torch.rand(T, generator=gen, device="cuda")
    got = mx.linear_cross_entropy_bwd(dloss, x, w, y, lse)
    z, dz = exact_dz(x, w, y, lse, dloss)
    _, bz = C.bars_of_logits(x, w)
    delta = 2.0 ** -16 + 2 * float(bz.max()) + 2.0 ** -20 + 2.0 ** -21 * float((z.abs() + lse.double().abs()[:, None]).max())
    bar = math.sqrt(2.0 ** -7 * delta)

    def apart(a, b):
        return float((a.bfloat16().double() - b.bfloat16().double()).norm() / b.norm())
    one = (dz / dloss.max()).bfloat16().double() * dloss.max()
    for g, want, planted in ((got[0], dz @ w.double(), one @ w.double()), (got[1], dz.t() @ x.double(), one.t() @ x.double())):
        assert apart(g, want) <= bar < apart(planted, want), (apart(g, want), bar, apart(planted, want))


@pytest.mark.parametrize("T", [40, 300, 1100])
def test_dz_is_relative_to_the_largest_weight(mx, T):
    import torch
    H, V = 256, 5000
    x, w, y = C.make(T, H, V, seed=T, ignored=0.0, scale=0.25, lean=0.0)
    _, lse = mx.linear_cross_entropy_fwd(x, w, y)
    dloss = torch.full((T,), (1 + 2.0 ** -8) / 1024, device="cuda")
    got = mx.linear_cross_entropy_bwd(dloss, x, w, y, lse)
    z, dz = exact_dz(x, w, y, lse, dloss)
    assert torch.exp(z - lse.double()[:, None]).max() < 2.0 ** -10
    bar = 2.0 ** -10 + 2.0 ** -8 / math.sqrt(T)
    plain = dz.bfloat16().double()

    def off(a, want):
        return abs(float((a.double() * want).sum() / (want * want).sum()) - 1)
    for g, want, planted in ((got[0], dz @ w.double(), plain @ w.double()), (got[1], dz.t() @ x.double(), plain.t() @ x.double())):
        assert off(g, want) <= bar < off(planted, want), (off(g, want), bar, off(planted, want))
