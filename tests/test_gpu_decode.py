"""The decode-time operators (moe_decode_fwd, nvfp4_moe_decode_fwd, mxfp8_matvec, nvfp4_matvec) against
their definitions in 64 bits.

Bars, from the arithmetic: the result is a bf16 rounding (half a bf16 step, 2^-9 of the value) of a
sum whose terms are off by at most delta of the largest magnitude among the 32 (16) activations of
their block, with fp32 accumulation behind it.  Against MXFP8 weights delta is 2^-16 for x and 2^-11 for
h (with the fp32 error of h's own sum), against NVFP4 weights 2^-13.  An element's error is therefore
bounded by 2^-8 |y| + delta * S, where S is the sum over the contraction of block maximum times
|weight|; the fp32 sums (in TMEM, of the K ranges and of h's inputs) stay below 2^-13 S for these
lengths.  Both terms are taken together with delta = 2^-10 for the MoE layer (two stages) and
delta = 2^-12 for one linear.
"""
import numpy as np
import pytest

from tests import _gpu as G

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


def weight(mx, fmt, M, K, seed):
    """(arguments for the call, 64-bit values [M, K]) of a random weight."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w = (0.02 * torch.randn((M, K), generator=gen, device="cuda")).bfloat16()
    if fmt == "mxfp8":
        q, sf, _, _ = mx.mxfp8_quantize(w, sf_layout=mx.SF_MMA)
        kt = (K // 32 + 3) // 4
        v = G.dequant(q.cpu().numpy(), G.sf_mma_to_compact(sf.cpu().numpy(), M, K // 32, kt))
        return (q, sf), torch.from_numpy(v).cuda()
    q, sf, amax = mx.nvfp4_quantize(w, sf_layout=mx.SF_MMA)
    s_enc = np.float32(2688.0) / amax.cpu().numpy()[0]
    v = G.nv_dequant(G.unpack_e2m1(q.cpu().numpy()), G.sf_mma_to_compact(sf.cpu().numpy(), M, K // 16, G.nv_kt(K)),
                     s_enc)
    return (q, sf, amax), torch.from_numpy(v).cuda()


def activations(T, K, seed, big=True):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, K), generator=gen, device="cuda")
    if big:
        x[:, :: max(1, K // 3)] *= 50.0
    return x.bfloat16()


def block_max(x, block):
    T, K = x.shape
    return x.abs().view(T, K // block, block).amax(-1).repeat_interleave(block, 1)


def check(y, ref, bound):
    import torch
    err = (y.double() - ref).abs()
    assert torch.isfinite(y.float()).all()
    bad = err > bound
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} elements off, worst {float((err / bound).max()):.3f} of the bar"


def matvec(mx, fmt, x, w, **kw):
    return mx.mxfp8_matvec(x, *w, **kw) if fmt == "mxfp8" else mx.nvfp4_matvec(x, w, **kw)


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
@pytest.mark.parametrize("T,K,N", [(1, 128, 128), (1, 4096, 384), (2, 256, 128), (7, 640, 256), (8, 2048, 128),
                                   (9, 384, 1280), (17, 1408, 256), (32, 512, 128), (33, 256, 256), (64, 1152, 640),
                                   (3, 14336, 256)])
def test_matvec(mx, fmt, T, K, N):
    import torch
    w, wv = weight(mx, fmt, N, K, seed=T + K)
    x = activations(T, K, seed=N)
    ws = torch.empty(mx.matvec_workspace_size(), dtype=torch.uint8, device="cuda")
    y = matvec(mx, fmt, x, w, workspace=ws)
    assert mx.mxfp8_check_device_error(ws) == (0, 0)
    ref = x.double() @ wv.t()
    S = block_max(x.double(), 32 if fmt == "mxfp8" else 16) @ wv.abs().t()
    check(y, ref, 2.0 ** -8 * ref.abs() + 2.0 ** -12 * S)
    assert torch.equal(y.view(torch.int16), matvec(mx, fmt, x, w).view(torch.int16)), "not reproducible"


def moe(mx, fmt, x, experts, gates, w1, w2, **kw):
    if fmt == "mxfp8":
        return mx.moe_decode_fwd(x, experts, gates, *w1, *w2, **kw)
    return mx.nvfp4_moe_decode_fwd(x, experts, gates, w1, w2, **kw)


def moe_ref(fmt, x, experts, gates, w1, w2, E, H, F):
    """(definition in 64 bits, bound on the error) per element."""
    import torch
    block = 32 if fmt == "mxfp8" else 16
    T = x.shape[0]
    ref = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    S = torch.zeros_like(ref)
    ids = experts.cpu().tolist()
    for t in range(T):
        for j, e in enumerate(ids[t]):
            if not 0 <= e < E:
                continue
            xt = x[t:t + 1].double()
            a, b = w1[e * 2 * F:e * 2 * F + F], w1[e * 2 * F + F:(e + 1) * 2 * F]
            g, u = xt @ a.t(), xt @ b.t()
            wt = 1.0 if gates is None else float(gates[t, j])
            s = g / (1 + torch.exp(-g))
            xm = block_max(xt, block)
            # |dh| <= |w| (|silu'| |dg| |u| + |silu| |du|), |silu'| <= 1.1
            dh = abs(wt) * (1.1 * (xm @ a.abs().t()) * u.abs() + s.abs() * (xm @ b.abs().t()))
            w2e = w2[e * H:(e + 1) * H]
            ref[t] += (wt * s * u @ w2e.t())[0]
            S[t] += ((block_max((wt * s * u), block) + dh * 2.0 ** -2) @ w2e.abs().t())[0]
    return ref, 2.0 ** -8 * ref.abs() + 2.0 ** -10 * S + 1e-30


CASES = [  # T, k, E, H, F, fraction of dropped choices, gates
    (1, 1, 1, 128, 128, 0.0, False), (1, 2, 8, 256, 384, 0.0, True), (5, 2, 4, 256, 512, 0.4, True),
    (8, 3, 16, 512, 128, 0.0, True), (9, 2, 3, 384, 256, 0.0, True), (31, 8, 64, 256, 128, 0.1, True),
    (32, 1, 2, 128, 1408, 0.0, False), (33, 2, 5, 256, 256, 0.0, True), (64, 4, 8, 512, 640, 0.2, True),
    (64, 2, 1024, 128, 128, 0.0, True), (4, 32, 40, 128, 128, 0.0, True), (3, 2, 2, 128, 128, 1.0, True),
]


@pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])
@pytest.mark.parametrize("T,k,E,H,F,drop,with_gates", CASES)
def test_moe(mx, fmt, T, k, E, H, F, drop, with_gates):
    import torch
    w1, v1 = weight(mx, fmt, E * 2 * F, H, seed=1)
    w2, v2 = weight(mx, fmt, E * H, F, seed=2)
    x = activations(T, H, seed=3)
    rng = np.random.default_rng(T * 131 + E)
    ids = np.stack([rng.permutation(E)[:k] if k <= E else rng.integers(0, E, k) for _ in range(T)]).astype(np.int32)
    gates = rng.uniform(0.05, 1.0, (T, k)).astype(np.float32)
    dropped = rng.random((T, k)) < drop
    ids[dropped] = -1
    gates[dropped] = np.nan          # whatever a dropped choice's gate holds, it is not read
    if T > 2 and drop > 0:
        ids[1] = -1
    ids, gates = G.to_dev(ids), (G.to_dev(gates) if with_gates else None)
    ws = torch.full((mx.moe_decode_workspace_size(T, k, H, F, E),), 0xFF, dtype=torch.uint8, device="cuda")
    out = moe(mx, fmt, x, ids, gates, w1, w2, workspace=ws)
    assert mx.mxfp8_check_device_error(ws) == (0, 0)
    ref, bound = moe_ref(fmt, x, ids, gates, v1, v2, E, H, F)
    check(out, ref, bound)
    if T > 2 and drop > 0:
        assert not out[1].view(torch.int16).any(), "a token without a choice gives zeros"
    again = moe(mx, fmt, x, ids, gates, w1, w2)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)), "not reproducible"
