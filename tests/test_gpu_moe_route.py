"""moe_route_fwd / moe_route_bwd against their formulas in 64 bits and against differences.

Bars, from the arithmetic (all in fp32): exp is within 2^-22 of its value, its argument l - top within 2^-24 of
itself, and x exp(-x) < 0.4, so a term of a token's sum is off by at most 2^-21 of the largest; the sum has at most 32
terms in sequence and five levels of a tree, 37 roundings of 2^-24.  So the sum is within 2^-18, lse within 2^-17
plus its own rounding, and a probability or gate within 2^-16 of its value (its logit at most 100 below the largest).
Column sums run over at most 512 tokens in sequence and a tree over the CTAs: 2^-14 of the sum.
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


def make(T, E, dtype, seed, closed=0.3, mask=True, scale=2.0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    l = scale * torch.randn((T, E), generator=gen, device="cuda")
    if closed > 0:
        l[torch.rand((T, E), generator=gen, device="cuda") < closed] = -math.inf
        l[torch.rand(T, generator=gen, device="cuda") < 0.05] = -math.inf
    m = None
    if mask:
        m = torch.rand(T, generator=gen, device="cuda") >= 0.25
        l[~m] = math.nan
    return l.to(torch.bfloat16 if dtype == "bf16" else torch.float32), m


def reference(logits, mask, k, normalize, spread):
    """(experts, gates, lse, counts, prob_sum, losses, p) from the definitions, choice by choice, on the host."""
    import torch
    l = logits.double().cpu()
    T, E = l.shape
    if mask is not None:
        l[~mask.cpu()] = -math.inf
    part = (l > -math.inf).any(1)
    lse = torch.full((T,), -math.inf, dtype=torch.float64)
    p = torch.zeros((T, E), dtype=torch.float64)
    lse[part] = torch.logsumexp(l[part], 1)
    p[part] = torch.exp(l[part] - lse[part][:, None])
    experts = torch.full((T, k), -1, dtype=torch.int32)
    gates = torch.zeros((T, k), dtype=torch.float64)
    counts = torch.zeros(E + 1, dtype=torch.int32)
    for t in range(T):
        row = sorted(((-float(v), e) for e, v in enumerate(l[t]) if v > -math.inf))[:k]
        for j in range(k):
            if j < len(row):
                experts[t, j], gates[t, j] = row[j][1], p[t, row[j][1]]
                counts[row[j][1]] += 1
            elif spread:
                experts[t, j] = (t * k + j) % E
        if normalize and row:
            gates[t] /= gates[t].sum()
    n = int(part.sum())
    counts[E] = n
    P = p.sum(0)
    balance = E * float((counts[:E].double() * P).sum()) / (max(n, 1) ** 2 * k)
    z = float((lse[part] ** 2).sum()) / max(n, 1)
    return experts, gates, lse, counts, P, torch.tensor([balance, z], dtype=torch.float64), p


def near(x, ref, bar, name):
    import torch
    x, ref = x.double().cpu(), ref.double().cpu()
    same = x == ref                       # infinities among them
    err = torch.where(same, torch.zeros_like(x), (x - ref).abs())
    assert (err <= bar).all(), f"{name}: worst {float((err / bar).max()):.3f} of the bar"


SHAPES = [(1, 1, 1), (1, 8, 2), (5, 3, 3), (7, 4, 1), (40, 5, 2), (33, 8, 8), (100, 16, 4), (70, 17, 6), (64, 32, 32),
          (300, 33, 5), (257, 64, 8), (50, 100, 8), (41, 128, 1), (20, 200, 32), (30, 256, 8), (19, 300, 3), (11, 512, 6),
          (9, 777, 32), (6, 1024, 4), (1500, 60, 6), (3000, 8, 2), (5000, 4, 3), (2500, 31, 31), (1300, 128, 8), (700, 256, 2),
          (400, 768, 20)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("dtype,normalize,spread", [("bf16", True, False), ("fp32", False, True), ("fp32", True, True)])
def test_forward(mx, T, E, k, dtype, normalize, spread):
    import torch
    logits, mask = make(T, E, dtype, seed=T * 31 + E * 7 + k)
    ws = torch.full((max(16, mx.moe_route_workspace_size(T, E, k)),), 255, dtype=torch.uint8, device="cuda")
    got = mx.moe_route_fwd(logits, k, token_mask=mask, normalize=normalize, spread=spread, workspace=ws)
    experts, gates, lse, counts, P, losses, _ = reference(logits, mask, k, normalize, spread)
    assert torch.equal(got[0].cpu(), experts) and torch.equal(got[3].cpu(), counts)
    near(got[1], gates, 2.0 ** -16 * gates + 1e-38, "gates")
    near(got[2], lse, 2.0 ** -17 + 2.0 ** -23 * lse.abs().nan_to_num(posinf=0.0, neginf=0.0), "lse")
    near(got[4], P, 2.0 ** -14 * P + 1e-38, "prob_sum")
    near(got[5], losses, 2.0 ** -13 * losses.abs() + 1e-30, "losses")


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("dtype,normalize,by_row,spread", [("bf16", True, True, True), ("fp32", False, False, False),
                                                          ("fp32", True, False, True)])
def test_backward(mx, T, E, k, dtype, normalize, by_row, spread):
    import torch
    logits, mask = make(T, E, dtype, seed=T * 5 + E * 3 + k)
    experts, gates, lse, counts, _, _ = mx.moe_route_fwd(logits, k, token_mask=mask, normalize=normalize, spread=spread)
    gen = torch.Generator(device="cuda").manual_seed(T + E)
    dg = torch.randn((T, k), generator=gen, device="cuda")
    dg[gates == 0] = math.nan                       # slots without a choice pass nothing on
    dp = 0.1 * torch.randn(E, generator=gen, device="cuda") / max(T, 1)
    dl = torch.tensor([0.7, -0.3], device="cuda")
    rows, given = None, dg
    if by_row:
        rows = torch.randperm(T * k, generator=gen, device="cuda").int().view(T, k)
        given = torch.empty(T * k, device="cuda")
        given[rows.view(-1).long()] = dg.view(-1)
    out = mx.moe_route_bwd(logits, experts, gates, lse, counts, dgates=given, dlosses=dl, row_of_slot=rows, dprob_sum=dp,
                           normalize=normalize)
    assert out.dtype == logits.dtype
    part = (lse > -math.inf)[:, None]
    p = torch.where(part, torch.exp(logits.double() - lse.double()[:, None]), 0.0)
    n = max(1, int(counts[E]))
    c = dp.double() + 0.7 * E * counts[:E].double() / (float(n) ** 2 * k)
    c = c[None, :].expand(T, E)
    a = torch.where(part, -0.6 * lse.double()[:, None] / n, 0.0)
    g, ids = gates.double(), experts.long().clamp(min=0)
    gd = torch.where(g > 0, g * dg.double(), 0.0)
    s, ms = gd.sum(1, keepdim=True), gd.abs().sum(1, keepdim=True)
    want = p * (c - (p * c).sum(1, keepdim=True) + a)
    mag = p * (c.abs() + (p * c.abs()).sum(1, keepdim=True) + a.abs())
    if normalize:
        want.scatter_add_(1, ids, gd - g * s)
        mag.scatter_add_(1, ids, gd.abs() + g * ms)
    else:
        want, mag = want - p * s, mag + p * ms
        want.scatter_add_(1, ids, gd)
        mag.scatter_add_(1, ids, gd.abs())
    half = torch.ldexp(torch.full_like(want, 0.505), torch.frexp(want)[1] - 8) if dtype == "bf16" else 0.0
    # a term is off by at most 2^-16 of its magnitude, as above
    near(out, want, (2.0 ** -15 * mag + half + 1e-38).cpu(), "dlogits")
    assert not out[(lse == -math.inf)].float().any()


@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_against_differences(mx, normalize):
    """Central differences in 64 bits of L = <dg, gates> + <dl, losses> + <dp, prob_sum>, the choices and their counts
    held fixed.  The kernel's fp32 gradient is within 2^-14 of the magnitudes; 1e-4 of the gradient's norm covers it,
    and the differences' own error of h^2 = 1e-10."""
    import torch
    T, E, k = 12, 9, 3
    logits, mask = make(T, E, "fp32", seed=3, closed=0.0, scale=1.0)
    experts, gates, lse, counts, _, _ = mx.moe_route_fwd(logits, k, token_mask=mask, normalize=normalize)
    gen = torch.Generator(device="cuda").manual_seed(9)
    dg = torch.randn((T, k), generator=gen, device="cuda")
    dp = torch.randn(E, generator=gen, device="cuda")
    dl = torch.tensor([2.0, 0.5], device="cuda")
    grad = mx.moe_route_bwd(logits, experts, gates, lse, counts, dgates=dg, dlosses=dl, dprob_sum=dp, normalize=normalize)
    n, f = int(mask.sum()), counts[:E].double()

    def loss(l):
        ls = torch.logsumexp(l, 1)
        p = torch.exp(l - ls[:, None])
        g = p.gather(1, experts[mask].long())
        if normalize:
            g = g / g.sum(1, keepdim=True)
        P = p.sum(0)
        return float((g * dg[mask].double()).sum() + 2.0 * E * (f * P).sum() / (n * n * k) + 0.5 * (ls * ls).mean() +
                     (P * dp.double()).sum())
    l = logits[mask].double()
    for _ in range(5):
        u = torch.randn(l.shape, generator=gen, device="cuda", dtype=torch.float64)
        h = 1e-5
        num = (loss(l + h * u) - loss(l - h * u)) / (2 * h)
        ana = float((grad[mask].double() * u).sum())
        assert abs(num - ana) <= 1e-4 * float(grad[mask].double().norm()) * 3, (num, ana)


@pytest.mark.parametrize("E", [4, 8, 31, 64, 200])
def test_ties_go_to_the_lowest_expert(mx, E):
    import torch
    k = min(4, E)
    l = torch.zeros((50, E), device="cuda")
    l[10:20, E - 1] = 1.0
    l[20:30] = -0.0
    l[30:40, ::2] = torch.finfo(torch.float32).min      # the type's lowest value is a logit like any other
    l[40:] = torch.finfo(torch.float32).min
    experts, gates, _, counts, _, _ = mx.moe_route_fwd(l, k)
    want = reference(l, None, k, True, False)
    assert torch.equal(experts.cpu(), want[0]) and torch.equal(counts.cpu(), want[3])
    near(gates, want[1], 2.0 ** -16 * want[1] + 1e-38, "gates")


@pytest.mark.parametrize("E", [8, 64])
def test_odd_logits_show_and_stay_in_their_token(mx, E):
    import torch
    logits, _ = make(40, E, "fp32", seed=1, closed=0.0, mask=False)
    clean = mx.moe_route_fwd(logits, 2)
    bad = logits.clone()
    bad[7, 3], bad[9, 1], bad[11, 0] = math.nan, math.inf, -math.nan
    experts, gates, lse, counts, _, losses = mx.moe_route_fwd(bad, 2)
    rows = torch.ones(40, dtype=torch.bool, device="cuda")
    rows[[7, 9, 11]] = False
    assert torch.equal(experts[rows], clean[0][rows]) and torch.equal(gates[rows], clean[1][rows])
    assert (experts[~rows] == -1).all() and not gates[~rows].any() and lse[~rows].isnan().all()
    assert int(counts[E]) == 40 and int(counts[:E].sum()) == 74 and losses.isnan().all()
    d = mx.moe_route_bwd(bad, experts, gates, lse, counts, dgates=torch.ones_like(gates))
    assert d[~rows].isnan().all() and d[rows].isfinite().all()


@pytest.mark.parametrize("T,E", [(0, 8), (5, 8), (2000, 8), (2000, 64)])
def test_no_token_takes_part(mx, T, E):
    import torch
    l = torch.full((T, E), math.nan, device="cuda")
    mask = torch.zeros(T, dtype=torch.bool, device="cuda")
    experts, gates, lse, counts, P, losses = mx.moe_route_fwd(l, 2, token_mask=mask)
    assert (experts == -1).all() and not gates.any() and (lse == -math.inf).all()
    assert not counts.any() and not P.any() and not losses.any()
    d = mx.moe_route_bwd(l, experts, gates, lse, counts, dgates=torch.full((T, 2), math.nan, device="cuda"),
                         dlosses=torch.ones(2, device="cuda"))
    assert d.shape == (T, E) and not d.any()


@pytest.mark.parametrize("E,k", [(8, 2), (8, 6), (64, 5), (300, 4), (1000, 9)])
def test_an_expert_listed_twice(mx, E, k):
    """The backward adds the shares of an expert that a token's list names more than once."""
    import torch
    T = 37
    gen = torch.Generator(device="cuda").manual_seed(E)
    logits = torch.randn((T, E), generator=gen, device="cuda")
    _, _, lse, counts, _, _ = mx.moe_route_fwd(logits, k)
    experts = torch.randint(0, max(1, E // 4), (T, k), generator=gen, device="cuda").int()
    experts[:, 1] = experts[:, 0]
    p = torch.exp(logits.double() - lse.double()[:, None])
    gates = p.gather(1, experts.long()).float()
    dg = torch.randn((T, k), generator=gen, device="cuda")
    got = mx.moe_route_bwd(logits, experts, gates, lse, counts, dgates=dg, normalize=False)
    gd = gates.double() * dg.double()
    want = -p * gd.sum(1, keepdim=True)
    mag = p * gd.abs().sum(1, keepdim=True)
    want.scatter_add_(1, experts.long(), gd)
    mag.scatter_add_(1, experts.long(), gd.abs())
    near(got, want, (2.0 ** -15 * mag + 1e-38).cpu(), "dlogits")
    again = mx.moe_route_bwd(logits, experts, gates, lse, counts, dgates=dg, normalize=False)
    assert torch.equal(got, again)


def test_counts_of_several_batches(mx):
    """The losses of two halves' summed counts: the two gradients are the whole batch's."""
    import torch
    logits, mask = make(600, 32, "fp32", seed=8)
    whole = mx.moe_route_fwd(logits, 4, token_mask=mask)
    halves = [mx.moe_route_fwd(logits[s].contiguous(), 4, token_mask=mask[s].contiguous())
              for s in (slice(0, 256), slice(256, 600))]
    counts = halves[0][3] + halves[1][3]
    assert torch.equal(counts, whole[3])
    dl = torch.tensor([1.0, 1.0], device="cuda")
    want = mx.moe_route_bwd(logits, *whole[:4], dlosses=dl)
    got = torch.cat([mx.moe_route_bwd(logits[s].contiguous(), *h[:3], counts, dlosses=dl)
                     for s, h in zip((slice(0, 256), slice(256, 600)), halves)])
    assert torch.equal(got, want)


def test_repeatable_captured_and_on_another_stream(mx):
    import torch
    logits, mask = make(5000, 64, "bf16", seed=4)
    ref = mx.moe_route_fwd(logits, 8, token_mask=mask)
    dl, dg = torch.ones(2, device="cuda"), torch.randn((5000, 8), device="cuda")
    ref_d = mx.moe_route_bwd(logits, *ref[:4], dgates=dg, dlosses=dl)

    def same(a, b):
        return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = mx.moe_route_fwd(logits, 8, token_mask=mask, stream=side)
    other_d = mx.moe_route_bwd(logits, *other[:4], dgates=dg, dlosses=dl, stream=side)
    side.synchronize()
    assert same(other, ref) and same([other_d], [ref_d])
    out = tuple(torch.empty_like(t) for t in ref)
    d = torch.empty_like(logits)
    ws = torch.empty(mx.moe_route_workspace_size(5000, 64, 8), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.moe_route_fwd(logits, 8, token_mask=mask, out=out, workspace=ws)
        mx.moe_route_bwd(logits, *out[:4], dgates=dg, dlosses=dl, out=d)
    for _ in range(2):
        for t in (*out, d):
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, ref) and same([d], [ref_d])
    logits.copy_(make(5000, 64, "bf16", seed=5, mask=False)[0])
    graph.replay()
    assert same(out, mx.moe_route_fwd(logits, 8, token_mask=mask))


def test_logits_at_odd_addresses(mx):
    import torch
    buf = torch.randn(33 * 7 + 1, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        b = buf.to(dtype)
        a, c = b[1:].view(33, 7), b[1:].clone().view(33, 7)
        assert a.data_ptr() % 16 != 0
        assert all(torch.equal(x, y) for x, y in zip(mx.moe_route_fwd(a, 3), mx.moe_route_fwd(c, 3)))
