"""residual_norm_fwd / residual_norm_bwd against their formulas in 64 bits and against differences.

Bars, from the arithmetic: values stored as bf16 are within half a bf16 step (8 significant bits) plus
the fp32 error of what was rounded; that error is below 2^-16 of the sum of the magnitudes of the
terms an element is made of (a few fp32 roundings of 2^-24 each, two row sums of up to 8192 terms added
in a tree, one reciprocal square root).  Column sums run over up to T / 152 rows in sequence and
then over 152 CTAs: below 2^-13 of the sum of the terms' magnitudes.
"""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from mxfp8_block_scaled_03_gb300 import build_ext
    build_ext.build()
    import mxfp8_block_scaled_03_gb300 as m
    m.lib()
    return m


EPS = 1e-6


def make(T, H, res, gate, post, seed, weights=True):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape):
        return torch.randn(shape, generator=gen, device="cuda")
    rt = torch.bfloat16 if res == "bf16" else torch.float32
    d = dict(y=(0.5 * rnd(T, H)).bfloat16(), res=(2 * rnd(T, H)).to(rt),
             w_post=1 + 0.2 * rnd(H) if post and weights else None, w_pre=1 + 0.2 * rnd(H) if weights else None,
             gate={"none": None, "channel": 0.5 * rnd(H), "token": torch.sigmoid(rnd(T, 1))}[gate],
             dn=(0.1 * rnd(T, H)).bfloat16(), dr=(0.1 * rnd(T, H)).to(rt))
    return d


def f64(t):
    return None if t is None else t.double()


def forward64(y, res, w_post, gate, w_pre, scale, post):
    import torch
    one = torch.ones((), dtype=torch.float64, device="cuda")
    rs1 = ((y * y).mean(1, keepdim=True) + EPS) ** -0.5 if post else torch.ones_like(y[:, :1])
    z = y * rs1 * (one if w_post is None else w_post)
    gz = z if gate is None else gate * z
    r = scale * res + gz
    rs2 = ((r * r).mean(1, keepdim=True) + EPS) ** -0.5
    return r, r * rs2 * (one if w_pre is None else w_pre), rs1, rs2, (scale * res).abs() + gz.abs()


def near(x, ref, mag, rel16, name):
    """|x - ref| within half a bf16 step where x is bf16, plus rel16 * mag."""
    import torch
    # bf16 step of values in [2^(e-1), 2^e): 2^(e-8); 1.01: the rounded value's exponent may be the next one
    half = torch.ldexp(torch.full_like(ref, 0.505), torch.frexp(ref)[1] - 8) if x.dtype == torch.bfloat16 else 0.0
    bar = rel16 * mag + half + 1e-30
    err = (x.double() - ref).abs()
    assert torch.isfinite(x.float()).all(), name
    assert (err <= bar).all(), f"{name}: worst {float((err / bar).max()):.3f} of the bar"


SHAPES = [(1, 8), (1, 4096), (3, 128), (5, 200), (17, 256), (40, 264), (7, 1000), (33, 1024), (9, 2056), (300, 2048),
          (2000, 512), (11, 4096), (4, 4104), (500, 5120), (13, 8192)]
KINDS = [("bf16", "channel", True, 1.0), ("fp32", "token", True, 0.75), ("bf16", "none", True, 1.0),
         ("fp32", "channel", False, 1.0), ("bf16", "token", False, -0.5)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("res,gate,post,scale", KINDS)
def test_forward_and_backward(mx, T, H, res, gate, post, scale):
    import torch
    d = make(T, H, res, gate, post, seed=T * 7 + H)
    r, n, stats = mx.residual_norm_fwd(d["y"], d["res"], w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"],
                                       res_scale=scale, post_norm=post, eps=EPS)
    y, wp, g, wn = f64(d["y"]), f64(d["w_post"]), f64(d["gate"]), f64(d["w_pre"])
    rr, rn, rs1, rs2, mag = forward64(y, f64(d["res"]), wp, g, wn, scale, post)
    near(r, rr, mag, 2.0 ** -16, "res_out")
    near(n, rn, mag * rs2 * wn.abs() + rn.abs(), 2.0 ** -16, "n")
    near(stats[0], rs1[:, 0], rs1[:, 0], 2.0 ** -16, "stats 0")
    near(stats[1], rs2[:, 0], rs2[:, 0], 2.0 ** -16, "stats 1")

    dy, dres, dwp, dg, dwn = mx.residual_norm_bwd(d["dn"], d["dr"], d["y"], r, stats, w_post=d["w_post"],
                                                  gate=d["gate"], w_pre=d["w_pre"], res_scale=scale, post_norm=post)
    s1, s2 = stats.double()[0][:, None], stats.double()[1][:, None]
    rh, a = r.double() * s2, f64(d["dn"]) * wn
    G = f64(d["dr"]) + s2 * (a - rh * (a * rh).mean(1, keepdim=True))
    mG = f64(d["dr"]).abs() + s2 * (a.abs() + rh.abs() * (a * rh).abs().mean(1, keepdim=True))
    near(dres, scale * G, abs(scale) * mG, 2.0 ** -16, "dres")
    yh = y * s1 if post else y
    z = yh * wp if post else yh
    one = torch.ones((), dtype=torch.float64, device="cuda")
    gg = one if g is None else g
    dz, mdz = gg * G, gg.abs() * mG
    if post:
        b, mb = dz * wp, mdz * wp.abs()
        near(dy, s1 * (b - yh * (b * yh).mean(1, keepdim=True)),
             s1 * (mb + yh.abs() * (mb * yh.abs()).mean(1, keepdim=True)), 2.0 ** -15, "dy")
        near(dwp, (dz * yh).sum(0), (mdz * yh.abs()).sum(0), 2.0 ** -13, "dw_post")
    else:
        near(dy, dz, mdz, 2.0 ** -15, "dy")
        assert dwp is None
    if gate == "channel":
        near(dg, (G * z).sum(0), (mG * z.abs()).sum(0), 2.0 ** -13, "dgate")
    elif gate == "token":
        near(dg, (G * z).sum(1, keepdim=True), (mG * z.abs()).sum(1, keepdim=True), 2.0 ** -13, "dgate")
    else:
        assert dg is None
    near(dwn, (f64(d["dn"]) * rh).sum(0), (f64(d["dn"]) * rh).abs().sum(0), 2.0 ** -13, "dw_pre")


def test_without_weights_and_without_residual_gradient(mx):
    import torch
    d = make(50, 768, "fp32", "none", True, seed=3, weights=False)
    r, n, stats = mx.residual_norm_fwd(d["y"], d["res"], eps=EPS)
    rr, rn, rs1, rs2, mag = forward64(f64(d["y"]), f64(d["res"]), None, None, None, 1.0, True)
    near(r, rr, mag, 2.0 ** -16, "res_out")
    near(n, rn, mag * rs2 + rn.abs(), 2.0 ** -16, "n")
    zero = torch.zeros_like(d["dr"])
    a = mx.residual_norm_bwd(d["dn"], None, d["y"], r, stats)
    b = mx.residual_norm_bwd(d["dn"], zero, d["y"], r, stats)
    assert a[2:] == (None, None, None)
    assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("res", ["bf16", "fp32"])
def test_in_place_and_repeatable(mx, res):
    import torch
    d = make(700, 2048, res, "channel", True, seed=9)
    kw = dict(w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"])
    r, n, stats = mx.residual_norm_fwd(d["y"], d["res"], **kw)
    buf = d["res"].clone()
    out = (buf, torch.empty_like(n), torch.empty_like(stats))
    mx.residual_norm_fwd(d["y"], buf, out=out, **kw)
    assert torch.equal(buf, r) and torch.equal(out[1], n) and torch.equal(out[2], stats)
    one = mx.residual_norm_bwd(d["dn"], d["dr"], d["y"], r, stats, **kw)
    two = mx.residual_norm_bwd(d["dn"], d["dr"], d["y"], r, stats, **kw)
    assert all(torch.equal(x, y) for x, y in zip(one, two))


def test_no_rows(mx):
    import torch
    H = 512
    y = torch.empty((0, H), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(H, device="cuda")
    r, n, stats = mx.residual_norm_fwd(y, y, w_post=w, gate=w, w_pre=w)
    assert r.shape == (0, H) and n.shape == (0, H)
    _, _, dwp, dg, dwn = mx.residual_norm_bwd(n, r, y, r, stats, w_post=w, gate=w, w_pre=w)
    assert not dwp.any() and not dg.any() and not dwn.any()


@pytest.mark.parametrize("gate,post", [("channel", True), ("token", True), ("none", False)])
def test_gradient_against_differences(mx, gate, post):
    """Directional derivatives of L = <dn, n> + <dr, res_out> by central differences in 64 bits.  The kernel's
    gradients differ from the formula's by bf16 roundings (2^-9 each, independent) and by res_out's rounding
    inside the norm's Jacobian: 1% of the derivative's scale covers both."""
    import torch
    T, H = 6, 256
    d = make(T, H, "fp32", gate, post, seed=21)
    kw = dict(w_post=d["w_post"], gate=d["gate"], w_pre=d["w_pre"])
    r, n, stats = mx.residual_norm_fwd(d["y"], d["res"], res_scale=0.9, post_norm=post, eps=EPS, **kw)
    grads = mx.residual_norm_bwd(d["dn"], d["dr"], d["y"], r, stats, res_scale=0.9, post_norm=post, **kw)
    ins = [f64(d["y"]), f64(d["res"]), f64(d["w_post"]), f64(d["gate"]), f64(d["w_pre"])]

    def loss(x):
        rr, nn, *_ = forward64(*x, 0.9, post)
        return float((f64(d["dn"]) * nn).sum() + (f64(d["dr"]) * rr).sum())
    gen = torch.Generator(device="cuda").manual_seed(5)
    for i, gr in enumerate(grads):
        if gr is None:
            continue
        for _ in range(3):
            u = torch.randn(ins[i].shape, generator=gen, device="cuda", dtype=torch.float64)
            h = 1e-5
            lo, hi = list(ins), list(ins)
            hi[i], lo[i] = ins[i] + h * u, ins[i] - h * u
            num = (loss(hi) - loss(lo)) / (2 * h)
            ana = float((gr.double() * u).sum())
            assert abs(num - ana) <= 0.01 * float((gr.double() * u).norm()) * 3, (i, num, ana)
