"""The decode-time operators hold on to their activations' bits: results that are small differences of two
activations, and the norm of the error on ordinary ones.  Inputs and bars of _decode_model, which derives them;
test_decode_precision_model shows on the CPU that they notice one missing piece or digit."""
import numpy as np
import pytest

from tests import _decode_model as M
from tests import _gpu as G
from tests import test_gpu_decode as D

pytestmark = pytest.mark.gpu

mx = D.mx
FORMATS = pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])


def exact_weight(mx, fmt, w):
    """Arguments for the call of a matrix both formats hold exactly; refused if it comes back changed."""
    import torch
    t = torch.from_numpy(w).cuda().bfloat16()
    rows, K = w.shape
    if fmt == "mxfp8":
        q, sf, _, _ = mx.mxfp8_quantize(t, sf_layout=mx.SF_MMA)
        v = G.dequant(q.cpu().numpy(), G.sf_mma_to_compact(sf.cpu().numpy(), rows, K // 32, (K // 32 + 3) // 4))
        assert (v == w).all()
        return q, sf
    q, sf, amax = mx.nvfp4_quantize(t, sf_layout=mx.SF_MMA)
    s_enc = np.float32(2688.0) / amax.cpu().numpy()[0]
    v = G.nv_dequant(G.unpack_e2m1(q.cpu().numpy()), G.sf_mma_to_compact(sf.cpu().numpy(), rows, K // 16, G.nv_kt(K)),
                     s_enc)
    assert (v == w).all()
    return q, sf, amax


def tokens(x):
    import torch
    return torch.from_numpy(x).cuda().bfloat16()


def within(y, ref, bar):
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= bar).all(), f"worst {float((err / bar).max()):.3f} of the bar, {int((err > bar).sum())} elements"


@FORMATS
@pytest.mark.parametrize("T,K,N", [(1, 512, 256), (5, 1408, 384), (12, 4096, 128), (23, 640, 512), (41, 2048, 128)])
def test_linear_keeps_small_differences(mx, fmt, T, K, N):
    x, w, a, b = M.linear_case(fmt, T, K, N, seed=K)
    y = D.matvec(mx, fmt, tokens(x), exact_weight(mx, fmt, w))
    ref = x @ w.T
    within(y, ref, M.linear_bar(fmt, x, ref, a, b))


@FORMATS
@pytest.mark.parametrize("E,H,F,repeat", [(3, 128, 384, 1), (2, 256, 1408, 1), (2, 128, 640, 13), (1, 128, 2048, 33),
                                          (4, 2048, 256, 2)])
def test_layer_keeps_small_differences(mx, fmt, E, H, F, repeat):
    """`repeat`: tokens per expert, copies of its one, so that groups of every size meet the same bar."""
    import torch
    x, gates, w1, w2, h, a, b = M.layer_case(fmt, E, H, F, seed=F)
    q1, q2 = exact_weight(mx, fmt, w1.reshape(-1, H)), exact_weight(mx, fmt, w2.reshape(-1, F))
    ids = torch.arange(E, dtype=torch.int32, device="cuda").repeat(repeat)[:, None].contiguous()
    gt = torch.from_numpy(np.tile(gates.astype(np.float32), repeat)[:, None]).cuda()
    y = D.moe(mx, fmt, tokens(np.tile(x, (repeat, 1))), ids, gt, q1, q2)
    ref = np.einsum("ehf,ef->eh", w2, h)
    within(y, np.tile(ref, (repeat, 1)), np.tile(M.layer_bar(fmt, h, ref, a, b), (repeat, 1)))


@FORMATS
@pytest.mark.parametrize("T,k,E,H,F,drop,with_gates", [c for c in D.CASES if c[5] < 1.0])
def test_error_norm_of_the_layer(mx, fmt, T, k, E, H, F, drop, with_gates):
    w1, v1 = D.weight(mx, fmt, E * 2 * F, H, seed=1)
    w2, v2 = D.weight(mx, fmt, E * H, F, seed=2)
    x = D.activations(T, H, seed=3)
    rng = np.random.default_rng(T * 131 + E)
    ids = np.stack([rng.permutation(E)[:k] if k <= E else rng.integers(0, E, k) for _ in range(T)]).astype(np.int32)
    ids[rng.random((T, k)) < drop] = -1
    gates = G.to_dev(rng.uniform(0.05, 1.0, (T, k)).astype(np.float32)) if with_gates else None
    ids = G.to_dev(ids)
    y = D.moe(mx, fmt, x, ids, gates, w1, w2)
    ref, _ = D.moe_ref(fmt, x, ids, gates, v1, v2, E, H, F)
    assert M.error_norm(y.double().cpu().numpy(), ref.cpu().numpy()) <= M.NORM_BAR


@FORMATS
@pytest.mark.parametrize("T,K,N", [(1, 4096, 384), (7, 640, 256), (33, 256, 256), (64, 1152, 640), (3, 14336, 256)])
def test_error_norm_of_a_linear(mx, fmt, T, K, N):
    w, wv = D.weight(mx, fmt, N, K, seed=T + K)
    x = D.activations(T, K, seed=N)
    y = D.matvec(mx, fmt, x, w)
    ref = x.double() @ wv.t()
    assert M.error_norm(y.double().cpu().numpy(), ref.cpu().numpy()) <= M.NORM_BAR
