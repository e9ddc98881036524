"""residual_norm_bwd against central differences of the formula in 64 bits, with bars from the roundings alone.

With a 32-bit residual only dy is rounded to bf16: an element is off by at most half a step, c = 2^-8 |dy|, evenly over
+-c, so that a sum of such errors with weights u has a spread of at most 2^-8 / sqrt(3) of the norm of dy * u; six of
those are allowed.  All gradients carry 32-bit errors: an element is made of a few terms no larger than the
largest gradient, each off by a few 2^-24 and by 2^-20 from the row sums (up to 256 terms) and the reciprocal square
root; 2^-17 of the largest gradient per element, and six spreads of their sum, give 2^-14 of it times the norm of u.  The
differences themselves are good to 1e-8 (step 1e-5, curvature and cancellation in 64 bits).
"""
import pytest

from tests import test_gpu_block_norm as B

pytestmark = pytest.mark.gpu

mx = B.mx


@pytest.mark.parametrize("T,H", [(1, 8), (6, 256), (19, 200)])
@pytest.mark.parametrize("gate,post,scale", [("channel", True, 0.9), ("token", True, 1.0), ("none", False, -0.5),
                                             ("token", False, 0.9)])
def test_directional_derivatives(mx, T, H, gate, post, scale):
    import torch
    d = B.make(T, H, "fp32", gate, post, seed=T + H)
    kw = dict(w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"])
    r, _, stats = mx.residual_norm_fwd(d["y"], d["res"], res_scale=scale, post_norm=post, eps=B.EPS, **kw)
    grads = mx.residual_norm_bwd(d["dn"], d["dr"], d["y"], r, stats, res_scale=scale, post_norm=post, **kw)
    ins = [B.f64(d[n]) for n in ("y", "res", "w_post", "gate", "w_pre")]

    def loss(x):
        rr, nn, *_ = B.forward64(*x, scale, post)
        return float((B.f64(d["dn"]) * nn).sum() + (B.f64(d["dr"]) * rr).sum())
    gen = torch.Generator(device="cuda").manual_seed(5)
    h = 1e-5
    for i, g in enumerate(grads):
        assert (g is None) == (ins[i] is None)
        if g is None:
            continue
        assert g.shape == ins[i].shape
        for _ in range(3):
            u = torch.randn(ins[i].shape, generator=gen, device="cuda", dtype=torch.float64)
            lo, hi = list(ins), list(ins)
            hi[i], lo[i] = ins[i] + h * u, ins[i] - h * u
            num, ana = (loss(hi) - loss(lo)) / (2 * h), float((g.double() * u).sum())
            bar = 2.0 ** -14 * float(g.abs().max()) * float(u.norm()) + 1e-8 * max(1.0, abs(num))
            if g.dtype == torch.bfloat16:
                bar += 6 * 2.0 ** -8 / 3 ** 0.5 * float((g.double() * u).norm())
            assert abs(num - ana) <= bar, (i, num, ana, bar)
