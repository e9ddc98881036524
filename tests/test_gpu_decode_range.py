"""Decode-time operators on activations of very different size in one row: a channel far above the others (a
"massive activation") whose weights are zero, so that the result is made of the small ones alone.

Bars: those of test_gpu_decode (derived there), whose sums leave the large channel out since its weights are zero,
plus 2^-31 of the row's largest magnitude per unit of weight, the absolute limit of the NVFP4 digits: a block's
scale reaches 2^-17 of the row's largest block, and the digits go 2^-14 below that.
"""
import numpy as np
import pytest

from tests import _gpu as G
from tests import test_gpu_decode as D

pytestmark = pytest.mark.gpu

mx = D.mx
FORMATS = pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])


def quantized(mx, fmt, w):
    """(arguments for the call, 64-bit values) of a bf16 matrix."""
    import torch
    M, K = w.shape
    if fmt == "mxfp8":
        q, sf, _, _ = mx.mxfp8_quantize(w, sf_layout=mx.SF_MMA)
        v = G.dequant(q.cpu().numpy(), G.sf_mma_to_compact(sf.cpu().numpy(), M, K // 32, (K // 32 + 3) // 4))
        return (q, sf), torch.from_numpy(v).cuda()
    q, sf, amax = mx.nvfp4_quantize(w, sf_layout=mx.SF_MMA)
    s_enc = np.float32(2688.0) / amax.cpu().numpy()[0]
    v = G.nv_dequant(G.unpack_e2m1(q.cpu().numpy()), G.sf_mma_to_compact(sf.cpu().numpy(), M, K // 16, G.nv_kt(K)),
                     s_enc)
    return (q, sf, amax), torch.from_numpy(v).cuda()


@FORMATS
@pytest.mark.parametrize("K,N", [(128, 128), (640, 256), (2048, 384), (17408, 128)])
def test_linear_beside_a_large_channel(mx, fmt, K, N):
    import torch
    powers = [0, 12, 15, 16, 17, 18, 19, 20, 23, 26, 40]
    gen = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn((len(powers), K), generator=gen, device="cuda")
    blk = K // 64 * 32                                   # 32 channels, one of them large
    for t, s in enumerate(powers):
        x[t, blk + (5 * t) % 32] = 1.5 * 2.0 ** s
    x = x.bfloat16()
    w = 0.02 * torch.randn((N, K), generator=gen, device="cuda")
    w[:, blk:blk + 32] = 0
    w, wv = quantized(mx, fmt, w.bfloat16())
    y = D.matvec(mx, fmt, x, w)
    ref = x.double() @ wv.t()
    S = D.block_max(x.double(), 32 if fmt == "mxfp8" else 16) @ wv.abs().t()
    low = x.double().abs().amax(1, keepdim=True) * 2.0 ** -31 * wv.abs().sum(1)
    D.check(y, ref, 2.0 ** -8 * ref.abs() + 2.0 ** -12 * S + (low if fmt == "nvfp4" else 0.0))


@FORMATS
def test_blocks_at_the_limit_of_the_scales(mx, fmt):
    """One small block beside the row's largest: from where its scale is the smallest there is, down to where its
    values leave the digits."""
    import torch
    K, N = 256, 128
    x = torch.zeros((24, K), device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    for t in range(24):
        x[t, 0] = 1.0
        x[t, 48:64] = torch.randn((16,), generator=gen, device="cuda") * 2.0 ** (-10 - t)
    x = x.bfloat16()
    w = torch.randn((N, K), generator=gen, device="cuda")
    w[:, :32] = 0
    w, wv = quantized(mx, fmt, w.bfloat16())
    y = D.matvec(mx, fmt, x, w)
    ref = x.double() @ wv.t()
    S = D.block_max(x.double(), 32 if fmt == "mxfp8" else 16) @ wv.abs().t()
    low = 2.0 ** -31 * wv[:, 48:64].abs().sum(1)
    D.check(y, ref, 2.0 ** -8 * ref.abs() + 2.0 ** -12 * S + (low if fmt == "nvfp4" else 0.0))


@FORMATS
def test_layer_on_tokens_with_a_large_channel(mx, fmt):
    """The same in front of a layer: W1's columns are zero at the large channel."""
    import torch
    T, k, E, H, F = 6, 2, 3, 640, 256
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((T, H), generator=gen, device="cuda")
    for t in range(T):
        x[t, 64 + 3 * t] = -(2.0 ** (13 + t))
    x = x.bfloat16()
    w1, w2 = 0.05 * torch.randn((E * 2 * F, H), generator=gen, device="cuda"), 0.02 * torch.randn((E * H, F), device="cuda")
    w1[:, 64:96] = 0
    w1, v1 = quantized(mx, fmt, w1.bfloat16())
    w2, v2 = quantized(mx, fmt, w2.bfloat16())
    ids = torch.rand((T, E), generator=gen, device="cuda").argsort(1)[:, :k].int().contiguous()
    y = D.moe(mx, fmt, x, ids, None, w1, w2)
    # The bar allows x 2^-12 of a block's largest value: 2^-14 of it are the digits', and 2^18 * 2^-31 = 2^-13 at most
    # comes from the large channel, to be held against blocks whose largest value is above 2/3.
    x[:, 64:96] = 0
    ref, bound = D.moe_ref(fmt, x, ids, None, v1, v2, E, H, F)
    D.check(y, ref, bound)


@FORMATS
@pytest.mark.parametrize("T,k,E,H,F", [(1, 1, 2, 256, 384), (7, 2, 3, 256, 1152), (20, 1, 1, 128, 640),
                                       (3, 2, 4, 4096, 512), (33, 2, 4, 256, 2048), (2, 2, 2, 512, 14336)])
@pytest.mark.parametrize("size", [1.0, 8.0, 64.0])
def test_layer_beside_a_large_channel(mx, fmt, T, k, E, H, F, size):
    """A channel of h far above the others (its gate and up rows follow the signs of a token), and zeros in W2's
    columns there."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(T * 64 + F)
    x = torch.randn((T, H), generator=gen, device="cuda")
    sign = torch.sign(x[0]) + (x[0] == 0)
    for t in range(1, T, 2):                             # half of the tokens: signs that agree by 3/4
        keep = torch.rand((H,), generator=gen, device="cuda") < 0.75
        x[t] = torch.where(keep, x[t].abs() * sign, x[t])
    x = x.bfloat16()
    w1 = 0.02 * torch.randn((E, 2, F, H), generator=gen, device="cuda")
    w2 = 0.02 * torch.randn((E, H, F), generator=gen, device="cuda")
    blk = F // 64 * 32
    w1[:, :, blk + 7] = 0.02 * size * sign
    w2[:, :, blk:blk + 32] = 0
    w1, v1 = quantized(mx, fmt, w1.view(-1, H).bfloat16())
    w2, v2 = quantized(mx, fmt, w2.view(-1, F).bfloat16())
    ids = torch.rand((T, E), generator=gen, device="cuda").argsort(1)[:, :k].int().contiguous()
    gates = 0.25 + torch.rand((T, k), generator=gen, device="cuda")
    y = D.moe(mx, fmt, x, ids, gates, w1, w2)
    ref, bound = D.moe_ref(fmt, x, ids, gates, v1, v2, E, H, F)
    if fmt == "nvfp4":
        for t in range(T):
            for j in range(k):
                e = int(ids[t, j])
                g, u = (x[t].double() @ v1[(2 * e + b) * F:(2 * e + b + 1) * F].t() for b in (0, 1))
                top = float((g / (1 + torch.exp(-g)) * u).abs().max() * gates[t, j])
                bound[t] += 2.0 ** -31 * top * v2[e * H:(e + 1) * H].abs().sum(1)
    D.check(y, ref, bound)
    again = D.moe(mx, fmt, x, ids, gates, w1, w2)
    assert torch.equal(y.view(torch.int16), again.view(torch.int16)), "not reproducible"
