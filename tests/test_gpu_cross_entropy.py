"""linear_cross_entropy_fwd / linear_cross_entropy_bwd against their formulas in 64 bits and against differences.

Bars, from the arithmetic.  A logit is a sum of H exact products accumulated in fp32, 16 of them at a time; every
accumulation is off by at most 2^-22 of the sum A of the products' magnitudes (the tensor core cuts off, it does not
round): (H / 16 + 8) 2^-22 A.  exp2 is within 2^-21, its argument within 2^-23 of the logit's and lse's magnitude; a sum of
exponentials has at most 32 + 8 + V / 128 terms in sequence: 2^-16 with V below 2^17.  dz is rounded to bf16, by 2^-8 of
its value; dx and dw are accumulated like the logits, over V and T terms, and rounded to bf16 (half a step).

Those bars are of the worst case.  The errors' norms are held too: independent roundings of dz by at most 2^-8 give
2^-8 / sqrt(3) of the result's norm (rows of w and of x close to orthogonal) and the results' own rounding at most
2^-8: together below 2^-7.
"""
import math

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


def make(T, H, V, seed, ignored=0.3, scale=1.0, lean=8.0, dtype=None):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn((V, H), generator=gen, device="cuda") / math.sqrt(H)).bfloat16()
    y = torch.randint(0, V, (T,), generator=gen, device="cuda")
    x = scale * torch.randn((T, H), generator=gen, device="cuda")
    if T and lean:
        x += lean * torch.rand((T, 1), generator=gen, device="cuda") * w[y].float()
    y[torch.rand(T, generator=gen, device="cuda") < ignored] = -100
    return x.bfloat16(), w, y.to(dtype or torch.int32)


def bars_of_logits(x, w):
    """(z, bar of z) in 64 bits."""
    X, W = x.double(), w.double()
    H = x.shape[1]
    return X @ W.t(), (H / 16 + 8) * 2.0 ** -22 * (X.abs() @ W.abs().t())


def check(got, ref, bar, name):
    err = (got.double() - ref).abs()
    assert got.isfinite().all(), name
    assert (err <= bar).all(), f"{name}: worst {float((err / bar).max()):.3f} of the bar"


def half_step(ref):
    import torch
    return torch.ldexp(torch.full_like(ref, 0.505), torch.frexp(ref)[1] - 8) + 1e-38


def check_forward(loss, lse, x, w, y):
    import torch
    z, bz = bars_of_logits(x, w)
    want = torch.logsumexp(z, 1)
    bar = bz.amax(1) + 2.0 ** -15 + 2.0 ** -21 * (want.abs() + z.abs().amax(1))
    check(lse, want, bar, "lse")
    at = y.long().clamp(min=0)[:, None]
    valid = y >= 0
    want = torch.where(valid, want - z.gather(1, at)[:, 0], 0.0)
    check(loss, want, torch.where(valid, bar + bz.gather(1, at)[:, 0], 0.0), "loss")


def check_backward(dx, dw, dloss, dlse, x, w, y, lse):
    import torch
    rows = torch.nonzero(y >= 0)[:, 0]
    assert not dx[y < 0].float().any() and dx.isfinite().all()
    X, W, t = x[rows].double(), w.double(), y[rows].long()
    z, bz = bars_of_logits(x[rows], w)
    L = lse[rows].double()[:, None]
    hot = dloss[rows].double()[:, None]
    rate = hot if dlse is None else hot + dlse[rows].double()[:, None]
    p = torch.exp(z - L)
    dz = rate * p
    err = (rate.abs() + 2.0 ** -23 * hot.abs()) * p * (2 * bz + 2.0 ** -20 + 2.0 ** -21 * (z.abs() + L.abs()))
    dz.scatter_add_(1, t[:, None], -hot)
    err.scatter_add_(1, t[:, None], 2.0 ** -22 * hot.abs())
    err += (dz.abs() + err) * 2.0 ** -8 + 1e-38
    T, V = len(rows), w.shape[0]
    want = dz @ W
    bar = err @ W.abs() + (V / 16 + 40) * 2.0 ** -22 * (dz.abs() @ W.abs())
    check(dx[rows], want, bar + half_step(want.abs() + bar), "dx")
    norm = float((dx[rows].double() - want).norm()), float(want.norm())
    want = dz.t() @ X
    bar = err.t() @ X.abs() + (T / 16 + 40) * 2.0 ** -22 * (dz.t().abs() @ X.abs())
    check(dw, want, bar + half_step(want.abs() + bar), "dw")
    norms = norm, (float((dw.double() - want).norm()), float(want.norm()))
    if V > 1:
        for e, n in norms:
            assert e <= 2.0 ** -7 * n + 1e-30, norms


SHAPES = [(1, 8, 1), (1, 8, 2), (3, 16, 100), (5, 64, 128), (2, 4096, 3001), (127, 72, 129), (128, 128, 256),
          (129, 200, 257), (200, 264, 1000), (300, 512, 5000), (257, 1032, 2049), (5, 1024, 32000), (64, 2056, 511),
          (32, 520, 3000), (33, 520, 3000),
          (1030, 256, 20011), (2500, 136, 9000), (777, 520, 30001), (256, 64, 50257), (8000, 256, 128), (3001, 40, 300),
          (1500, 1024, 1000), (40, 128, 130), (65, 64, 128), (1024, 512, 8192), (1024, 2056, 1024), (1025, 512, 1100),
          (512, 8, 20000), (400, 512, 256), (100, 2048, 32000), (1000, 1448, 3600)]


@pytest.mark.parametrize("T,H,V", SHAPES)
def test_forward_and_backward(mx, T, H, V):
    import torch
    x, w, y = make(T, H, V, seed=T + H + V)
    if not (y >= 0).any():
        y[0] = 0
    ws = torch.full((mx.linear_cross_entropy_workspace_size(T, H, V),), 255, dtype=torch.uint8, device="cuda")
    loss, lse = mx.linear_cross_entropy_fwd(x, w, y, workspace=ws)
    assert mx.mxfp8_check_device_error(ws) == (0, 0)
    check_forward(loss, lse, x, w, y)
    gen = torch.Generator(device="cuda").manual_seed(1)
    dloss = torch.rand(T, generator=gen, device="cuda") / T
    dlse = 0.1 * torch.randn(T, generator=gen, device="cuda") / T
    ws = torch.full((mx.linear_cross_entropy_bwd_workspace_size(T, H, V),), 255, dtype=torch.uint8, device="cuda")
    dx, dw = mx.linear_cross_entropy_bwd(dloss, x, w, y, lse, dlse=dlse, workspace=ws)
    assert mx.mxfp8_check_device_error(ws) == (0, 0)
    check_backward(dx, dw, dloss, dlse, x, w, y, lse)


@pytest.mark.parametrize("T,H,V,ignored", [(16400, 72, 20001, 0.0), (1000, 16, 300001, 0.2)])
def test_several_pieces_of_the_vocabulary(mx, T, H, V, ignored):
    """dz of more than 2^28 elements: the vocabulary takes two pieces; dx is the sum over them."""
    import torch
    x, w, y = make(T, H, V, seed=2, ignored=ignored)
    loss, lse = mx.linear_cross_entropy_fwd(x, w, y)
    check_forward(loss, lse, x, w, y)
    dloss = torch.full((T,), 1.0 / T, device="cuda")
    ws = torch.full((mx.linear_cross_entropy_bwd_workspace_size(T, H, V),), 255, dtype=torch.uint8, device="cuda")
    dx, dw = mx.linear_cross_entropy_bwd(dloss, x, w, y, lse, workspace=ws)
    check_backward(dx, dw, dloss, None, x, w, y, lse)


@pytest.mark.parametrize("T,V", [(40, 700), (300, 5000), (1000, 2049), (1100, 20000)])
def test_rows_without_a_target_hold_anything(mx, T, V):
    """NaN and infinities in x, lse, dloss and dlse of rows that take no part reach nothing."""
    import torch
    H = 320
    x, w, y = make(T, H, V, seed=5)
    loss, lse = mx.linear_cross_entropy_fwd(x, w, y)
    dloss, dlse = torch.rand(T, device="cuda") / T, torch.rand(T, device="cuda") / T
    clean = mx.linear_cross_entropy_bwd(dloss, x, w, y, lse, dlse=dlse)
    off = y < 0
    for t, v in ((x, math.nan), (lse, math.inf), (dloss, math.nan), (dlse, -math.inf)):
        t[off] = v
    loss2, _ = mx.linear_cross_entropy_fwd(x, w, y)
    assert torch.equal(loss2, loss) and not loss[off].any()
    dirty = mx.linear_cross_entropy_bwd(dloss, x, w, y, lse, dlse=dlse)
    assert all(torch.equal(a, b) for a, b in zip(clean, dirty)) and not dirty[0][off].any()


@pytest.mark.parametrize("T", [0, 1, 300, 1100])
def test_no_row_takes_part(mx, T):
    import torch
    x = torch.full((T, 64), math.nan, dtype=torch.bfloat16, device="cuda")
    w = torch.randn((500, 64), device="cuda").bfloat16()
    y = torch.full((T,), -1, device="cuda")
    loss, lse = mx.linear_cross_entropy_fwd(x, w, y)
    assert loss.shape == lse.shape == (T,) and not loss.any()
    out = torch.full_like(x, 3.0), torch.full_like(w, 3.0)
    dx, dw = mx.linear_cross_entropy_bwd(torch.ones(T, device="cuda"), x, w, y, lse, out=out)
    assert dx is out[0] and not dx.any() and not dw.any()


@pytest.mark.parametrize("T", [50, 300, 1100])
def test_targets_of_both_types_and_out_of_range(mx, T):
    import torch
    H, V = 64, 300
    x, w, y = make(T, H, V, seed=7, dtype=torch.int64)
    a, b = mx.linear_cross_entropy_fwd(x, w, y), mx.linear_cross_entropy_fwd(x, w, y.int())
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    dloss = torch.rand(T, device="cuda")
    ga, gb = (mx.linear_cross_entropy_bwd(dloss, x, w, t, a[1]) for t in (y, y.int()))
    assert all(torch.equal(p, q) for p, q in zip(ga, gb))
    for far in (V, V + 5, 1 << 40):
        t = y.clone()
        t[3] = far
        ws = torch.empty(mx.linear_cross_entropy_workspace_size(T, H, V), dtype=torch.uint8, device="cuda")
        loss, lse = mx.linear_cross_entropy_fwd(x, w, t, workspace=ws)
        assert mx.mxfp8_check_device_error(ws)[0] == mx.ERR_INVALID_ARG
        assert loss[3].isnan() and loss.isnan().sum() == 1 and torch.equal(lse, a[1])
        ws = torch.empty(mx.linear_cross_entropy_bwd_workspace_size(T, H, V), dtype=torch.uint8, device="cuda")
        got = mx.linear_cross_entropy_bwd(dloss, x, w, t, lse, workspace=ws)
        assert mx.mxfp8_check_device_error(ws)[0] == mx.ERR_INVALID_ARG
        t[3] = -1
        want = mx.linear_cross_entropy_bwd(dloss, x, w, t, lse)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    loss, _ = mx.linear_cross_entropy_fwd(x, w, torch.full((T,), -(1 << 40), device="cuda"))
    assert not loss.any()


@pytest.mark.parametrize("scale", [0.0, 30.0, 1000.0])
def test_flat_and_peaked_rows(mx, scale):
    """All logits equal; and logits of hundreds, where one probability is 1 and the others vanish."""
    import torch
    T, H, V = 70, 128, 1000
    x, w, y = make(T, H, V, seed=11, scale=scale, lean=0.0, ignored=0.1)
    loss, lse = mx.linear_cross_entropy_fwd(x, w, y)
    check_forward(loss, lse, x, w, y)
    if scale == 0.0:
        assert (lse - math.log(V)).abs().max() < 1e-5
    y = torch.where(y < 0, y, (x.float() @ w.float().t()).argmax(1).int())   # the likeliest as targets, half of them
    y[::2] = (y[::2] + 1).clamp(max=V - 1)
    dloss = torch.ones(T, device="cuda")
    dx, dw = mx.linear_cross_entropy_bwd(dloss, x, w, y, lse)
    assert dx.isfinite().all() and dw.isfinite().all()
    if scale < 1000.0:
        check_backward(dx, dw, dloss, None, x, w, y, lse)


def test_gradient_against_differences(mx):
    """Central differences in 64 bits of L = <dloss, loss> + <dlse, lse>.  The kernel's gradient has roundings of 2^-8,
    independent of the direction: 2% of the gradient's norm covers them."""
    import torch
    T, H, V = 24, 64, 500
    x, w, y = make(T, H, V, seed=13, ignored=0.2)
    _, lse = mx.linear_cross_entropy_fwd(x, w, y)
    gen = torch.Generator(device="cuda").manual_seed(2)
    dloss, dlse = torch.rand(T, generator=gen, device="cuda"), 0.2 * torch.rand(T, generator=gen, device="cuda")
    grads = mx.linear_cross_entropy_bwd(dloss, x, w, y, lse, dlse=dlse)
    valid = y >= 0

    def loss(a, b):
        z = a @ b.t()
        ls = torch.logsumexp(z, 1)
        ce = ls - z.gather(1, y.long().clamp(min=0)[:, None])[:, 0]
        return float(((dloss * ce + dlse * ls) * valid).sum())
    ins = [x.double(), w.double()]
    for i, g in enumerate(grads):
        for _ in range(3):
            u = torch.randn(ins[i].shape, generator=gen, device="cuda", dtype=torch.float64)
            hi, lo = list(ins), list(ins)
            hi[i], lo[i] = ins[i] + 1e-5 * u, ins[i] - 1e-5 * u
            num = (loss(*hi) - loss(*lo)) / 2e-5
            ana = float((g.double() * u).sum())
            assert abs(num - ana) <= 0.02 * float(g.double().norm()), (i, num, ana)


@pytest.mark.parametrize("T,H,V", [(30, 256, 3000), (300, 256, 3000), (1200, 256, 20000)])
def test_repeatable_captured_and_on_another_stream(mx, T, H, V):
    import torch
    x, w, y = make(T, H, V, seed=17)
    dloss = torch.rand(T, device="cuda") / T
    loss, lse = mx.linear_cross_entropy_fwd(x, w, y)
    ref = (loss, lse, *mx.linear_cross_entropy_bwd(dloss, x, w, y, lse))

    def same(a, b):
        return all(torch.equal(p, q) for p, q in zip(a, b))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    f = mx.linear_cross_entropy_fwd(x, w, y, stream=side)
    got = (*f, *mx.linear_cross_entropy_bwd(dloss, x, w, y, f[1], stream=side))
    side.synchronize()
    assert same(got, ref)
    out = tuple(torch.empty_like(t) for t in ref)
    wf = torch.empty(mx.linear_cross_entropy_workspace_size(T, H, V), dtype=torch.uint8, device="cuda")
    wb = torch.empty(mx.linear_cross_entropy_bwd_workspace_size(T, H, V), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.linear_cross_entropy_fwd(x, w, y, out=out[:2], workspace=wf)
        mx.linear_cross_entropy_bwd(dloss, x, w, y, out[1], out=out[2:], workspace=wb)
    for seed in (17, 18):
        x2, w2, y2 = make(T, H, V, seed=seed)
        for a, b in ((x, x2), (w, w2), (y, y2)):
            a.copy_(b)
        for t in out:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        f = mx.linear_cross_entropy_fwd(x, w, y)
        assert same(out, (*f, *mx.linear_cross_entropy_bwd(dloss, x, w, y, f[1])))


def test_neighbours_of_the_outputs_are_left_alone(mx):
    import torch
    T, H, V = 37, 72, 203
    x, w, y = make(T, H, V, seed=23)
    bufs = [torch.full((n + 64,), 9.0, dtype=d, device="cuda") for n, d in
            ((T, torch.float32), (T, torch.float32), (T * H, torch.bfloat16), (V * H, torch.bfloat16))]
    loss, lse = bufs[0][32:32 + T], bufs[1][32:32 + T]
    dx, dw = bufs[2][32:32 + T * H].view(T, H), bufs[3][32:32 + V * H].view(V, H)
    mx.linear_cross_entropy_fwd(x, w, y, out=(loss, lse))
    mx.linear_cross_entropy_bwd(torch.ones(T, device="cuda"), x, w, y, lse, out=(dx, dw))
    for b, n in zip(bufs, (T, T, T * H, V * H)):
        assert (b[:32] == 9).all() and (b[32 + n:] == 9).all()


@pytest.mark.parametrize("T", [30, 300, 1100])
@pytest.mark.parametrize("loss_scale,lse_scale", [(0.0, 1.0), (1.0, 0.0), (0.0, 0.0), (1e-30, 1e10), (1e10, 1e-30), (1e-38, 1e-39)])
def test_weights_of_any_size(mx, T, loss_scale, lse_scale):
    """dloss alone, dlse alone, neither, and each far above the other: dx and dw scale with them."""
    import torch
    H, V = 128, 700
    x, w, y = make(T, H, V, seed=31)
    _, lse = mx.linear_cross_entropy_fwd(x, w, y)
    gen = torch.Generator(device="cuda").manual_seed(3)
    dloss = loss_scale * (0.5 + torch.rand(T, generator=gen, device="cuda"))
    dlse = lse_scale * (0.5 + torch.rand(T, generator=gen, device="cuda"))
    dx, dw = mx.linear_cross_entropy_bwd(dloss, x, w, y, lse, dlse=dlse)
    if loss_scale == lse_scale == 0.0:
        assert not dx.any() and not dw.any()
        return
    scale = max(loss_scale, lse_scale)
    rows = torch.nonzero(y >= 0)[:, 0]
    X, W = x[rows].double(), w.double()
    dz = (dloss + dlse.double())[rows][:, None] * torch.exp(X @ W.t() - lse[rows].double()[:, None])
    dz.scatter_add_(1, y[rows].long()[:, None], -dloss[rows].double()[:, None])
    for got, want in ((dx[rows], dz @ W), (dw, dz.t() @ X)):
        # by the norms (see above), and below 2^-126 by the results' own steps of 2^-133
        assert got.isfinite().all()
        err = float((got.double() - want).norm())
        assert err <= 2.0 ** -7 * float(want.norm()) + 2.0 ** -134 * want.numel() ** 0.5, (scale, err)


def test_one_row_with_a_weight_of_nan_stays_its_own(mx):
    """NaN in dloss of a row that takes part: NaN in its dx and in dw, nothing in the other rows of dx."""
    import torch
    for T in (20, 200, 1100):
        x, w, y = make(T, 64, 300, seed=4, ignored=0.0)
        _, lse = mx.linear_cross_entropy_fwd(x, w, y)
        dloss = torch.ones(T, device="cuda")
        clean, _ = mx.linear_cross_entropy_bwd(dloss, x, w, y, lse)
        dloss[3] = math.nan
        dx, dw = mx.linear_cross_entropy_bwd(dloss, x, w, y, lse)
        keep = torch.arange(T, device="cuda") != 3
        assert dx[3].isnan().all() and dw.isnan().all() and torch.equal(dx[keep], clean[keep])


@pytest.mark.parametrize("T", [20, 200])
def test_more_than_four_gigabytes_of_weights(mx, T):
    """V * H past 2^31 elements: rows of dw and logits beyond that offset."""
    import torch
    H, V = 2056, (1 << 20) + 77
    gen = torch.Generator(device="cuda").manual_seed(6)
    w = torch.empty((V, H), dtype=torch.bfloat16, device="cuda")
    for r in range(0, V, 65536):
        w[r:r + 65536] = torch.randn((min(65536, V - r), H), generator=gen, device="cuda") / math.sqrt(H)
    y = torch.randint(0, V, (T,), generator=gen, device="cuda")
    y[:4] = torch.tensor([V - 1, V - 77, 1 << 20, 0], device="cuda")
    x = (torch.randn((T, H), generator=gen, device="cuda") + 8.0 * w[y].float()).bfloat16()
    loss, lse = mx.linear_cross_entropy_fwd(x, w, y)
    m = torch.full((T,), -math.inf, dtype=torch.float64, device="cuda")
    for r in range(0, V, 131072):
        m = torch.logaddexp(m, torch.logsumexp(x.double() @ w[r:r + 131072].double().t(), 1))
    zy = (x.double() * w[y].double()).sum(1)
    bar = 2.0 ** -15 + (H / 16 + 8) * 2.0 ** -22 * 4 * math.sqrt(H)   # sum of |x w|: below 4 sqrt(H) here
    assert (lse.double() - m).abs().max() <= bar and (loss.double() - (m - zy)).abs().max() <= 2 * bar
    dloss = torch.full((T,), 1.0 / T, device="cuda")
    dx, dw = mx.linear_cross_entropy_bwd(dloss, x, w, y, lse)
    want = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for r in range(0, V, 131072):
        W = w[r:r + 131072].double()
        dz = torch.exp(x.double() @ W.t() - lse.double()[:, None]) / T
        hit = torch.nonzero((y >= r) & (y < r + len(W)))[:, 0]
        dz[hit, y[hit] - r] -= 1.0 / T
        want += dz @ W
        if r in (0, 1 << 20) or r + len(W) == V:
            ref = dz.t() @ x.double()
            assert (dw[r:r + len(W)].double() - ref).norm() <= 2.0 ** -7 * ref.norm()
    assert (dx.double() - want).norm() <= 2.0 ** -7 * want.norm()
