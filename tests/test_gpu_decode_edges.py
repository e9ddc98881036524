"""The decode-time operators at their edges: non-finite and extreme activations, choices that are
dropped, repeated or out of range, calls without tokens, other streams, graphs, refused tensors, and a
pipeline wait that runs out.  Bars as in test_gpu_decode (derived there)."""
import os
import subprocess
import sys

import numpy as np
import pytest

from tests import _gpu as G
from tests import test_gpu_decode as D

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

mx = D.mx
FORMATS = pytest.mark.parametrize("fmt", ["mxfp8", "nvfp4"])


@FORMATS
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_activations_stay_in_their_row(mx, fmt, value):
    import torch
    T, K, N = 5, 512, 256
    w, _ = D.weight(mx, fmt, N, K, seed=1)
    x = D.activations(T, K, seed=2)
    clean = D.matvec(mx, fmt, x, w)
    x[3, 77] = value
    y = D.matvec(mx, fmt, x, w)
    assert not torch.isfinite(y[3].float()).any()
    keep = [0, 1, 2, 4]
    assert torch.equal(y[keep].view(torch.int16), clean[keep].view(torch.int16))

    E, H, F, k = 4, 256, 256, 2
    w1, _ = D.weight(mx, fmt, E * 2 * F, H, seed=3)
    w2, _ = D.weight(mx, fmt, E * H, F, seed=4)
    x = D.activations(T, H, seed=5)
    ids = G.to_dev(np.array([[0, 1], [1, 2], [1, 3], [1, 0], [-1, 2]], dtype=np.int32))
    clean = D.moe(mx, fmt, x, ids, None, w1, w2)
    x[3, 11] = value
    y = D.moe(mx, fmt, x, ids, None, w1, w2)
    assert not torch.isfinite(y[3].float()).any()
    assert torch.equal(y[keep].view(torch.int16), clean[keep].view(torch.int16))


@FORMATS
def test_token_without_choices_ignores_its_activations(mx, fmt):
    import torch
    E, H, F = 4, 256, 256
    w1, _ = D.weight(mx, fmt, E * 2 * F, H, seed=3)
    w2, _ = D.weight(mx, fmt, E * H, F, seed=4)
    x = D.activations(3, H, seed=5)
    x[1] = float("nan")
    gates = torch.tensor([[0.5], [float("nan")], [0.25]], device="cuda")
    ids = G.to_dev(np.array([[0], [-7], [3]], dtype=np.int32))
    y = D.moe(mx, fmt, x, ids, gates, w1, w2)
    assert torch.isfinite(y.float()).all() and not y[1].view(torch.int16).any() and y[0].any() and y[2].any()


@FORMATS
@pytest.mark.parametrize("exponent", [-90, -20, 60])
def test_scale_of_the_activations_carries_through(mx, fmt, exponent):
    """Every power of two in reach moves the result by exactly that power: block scales are powers of two."""
    import torch
    T, K, N = 3, 640, 256
    w, _ = D.weight(mx, fmt, N, K, seed=6)
    x = D.activations(T, K, seed=7, big=False)
    x = torch.where(x.abs() < 2.0 ** -6, torch.zeros_like(x), x)   # keeps every block above 2^-100 at 2^-90
    y = D.matvec(mx, fmt, x, w)
    z = D.matvec(mx, fmt, torch.ldexp(x.float(), torch.tensor(exponent)).bfloat16(), w)
    assert torch.equal(torch.ldexp(y.float(), torch.tensor(exponent)), z.float())


@FORMATS
def test_zero_and_uneven_blocks(mx, fmt):
    import torch
    T, K, N = 4, 1024, 384
    w, wv = D.weight(mx, fmt, N, K, seed=8)
    x = D.activations(T, K, seed=9, big=False)
    x[0] = 0
    x[1, 64:] = 0
    x[2, :512] *= 2.0 ** -30      # blocks far below the row's largest
    x[3, ::16] *= 2.0 ** 20
    y = D.matvec(mx, fmt, x, w)
    ref = x.double() @ wv.t()
    assert not y[0].any()
    S = D.block_max(x.double(), 32 if fmt == "mxfp8" else 16) @ wv.abs().t()
    # NVFP4: blocks below 2^-17 of the row's largest value are dropped
    S = S + x.double().abs().amax(1, keepdim=True) * 2.0 ** -5 * wv.abs().sum(1)
    D.check(y, ref, 2.0 ** -8 * ref.abs() + 2.0 ** -12 * S + 1e-30)


@FORMATS
def test_repeated_choices_add_their_weights(mx, fmt):
    import torch
    T, k, E, H, F = 6, 5, 3, 256, 256
    w1, v1 = D.weight(mx, fmt, E * 2 * F, H, seed=1)
    w2, v2 = D.weight(mx, fmt, E * H, F, seed=2)
    x = D.activations(T, H, seed=3)
    rng = np.random.default_rng(4)
    ids, gates = G.to_dev(rng.integers(0, E, (T, k)).astype(np.int32)), G.to_dev(rng.random((T, k), dtype=np.float32))
    for g in (gates, None):
        y = D.moe(mx, fmt, x, ids, g, w1, w2)
        ref, bound = D.moe_ref(fmt, x, ids, g, v1, v2, E, H, F)
        D.check(y, ref, bound)


@FORMATS
def test_expert_out_of_range_is_reported_and_skipped(mx, fmt):
    import torch
    E, H, F = 4, 256, 256
    w1, _ = D.weight(mx, fmt, E * 2 * F, H, seed=1)
    w2, _ = D.weight(mx, fmt, E * H, F, seed=2)
    x = D.activations(2, H, seed=3)
    ws = torch.empty(mx.moe_decode_workspace_size(2, 2, H, F, E), dtype=torch.uint8, device="cuda")
    good = D.moe(mx, fmt, x, G.to_dev(np.array([[1, -1], [-1, 2]], dtype=np.int32)), None, w1, w2, workspace=ws)
    assert mx.mxfp8_check_device_error(ws) == (0, 0)
    y = D.moe(mx, fmt, x, G.to_dev(np.array([[1, 4], [2 ** 31 - 1, 2]], dtype=np.int32)), None, w1, w2, workspace=ws)
    st, bits = mx.mxfp8_check_device_error(ws)
    assert st == mx.ERR_INVALID_ARG and bits == 4
    assert torch.equal(y.view(torch.int16), good.view(torch.int16))


@FORMATS
def test_no_tokens(mx, fmt):
    import torch
    E, H, F = 2, 256, 256
    w1, _ = D.weight(mx, fmt, E * 2 * F, H, seed=1)
    w2, _ = D.weight(mx, fmt, E * H, F, seed=2)
    ws = torch.full((mx.moe_decode_workspace_size(0, 2, H, F, E),), 0xFF, dtype=torch.uint8, device="cuda")
    y = D.moe(mx, fmt, torch.empty((0, H), dtype=torch.bfloat16, device="cuda"),
              torch.empty((0, 2), dtype=torch.int32, device="cuda"), None, w1, w2, workspace=ws)
    assert y.shape == (0, H) and mx.mxfp8_check_device_error(ws) == (0, 0)
    assert D.matvec(mx, fmt, torch.empty((0, F), dtype=torch.bfloat16, device="cuda"), w2).shape == (0, E * H)


@FORMATS
def test_graph_replay_and_side_stream(mx, fmt):
    """Captured on a side stream, replayed on changed inputs, against the same calls made directly."""
    import torch
    T, k, E, H, F = 3, 2, 8, 256, 384
    w1, _ = D.weight(mx, fmt, E * 2 * F, H, seed=1)
    w2, _ = D.weight(mx, fmt, E * H, F, seed=2)
    x, ids = D.activations(T, H, seed=3), torch.empty((T, k), dtype=torch.int32, device="cuda")
    gates = torch.rand((T, k), device="cuda")
    out, out2 = (torch.empty((T, H), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.empty(mx.moe_decode_workspace_size(T, k, H, F, E), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(mx.matvec_workspace_size(T, F), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(0)

    def route():
        ids.copy_(torch.from_numpy(np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)))

    def step():
        D.moe(mx, fmt, x, ids, gates, w1, w2, out=out, workspace=ws)
        D.matvec(mx, fmt, torch.cat([out, out], 1)[:, :F].contiguous(), w2, workspace=ws2)
    route()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        D.moe(mx, fmt, x, ids, gates, w1, w2, out=out, workspace=ws)
    for _ in range(3):
        route()
        x.copy_(D.activations(T, H, seed=int(rng.integers(1000))))
        g.replay()
        D.moe(mx, fmt, x, ids, gates, w1, w2, out=out2)
        assert torch.equal(out.view(torch.int16), out2.view(torch.int16))


def test_refused_tensors(mx):
    import torch
    K, N = 256, 128
    w, _ = D.weight(mx, "nvfp4", N, K, seed=1)
    w8, _ = D.weight(mx, "mxfp8", N, K, seed=1)
    x = D.activations(2, K, seed=2)
    for bad in (x.float(), x.cpu(), x.t().contiguous().t(), x[:, :128].contiguous()):
        with pytest.raises(ValueError):
            mx.nvfp4_matvec(bad, w)
        with pytest.raises(ValueError):
            mx.mxfp8_matvec(bad, *w8)
    with pytest.raises(ValueError):
        mx.nvfp4_matvec(x, (w[0], w[1][:-1], w[2]))
    with pytest.raises(ValueError):
        mx.nvfp4_matvec(x, w, out=torch.empty((2, N), device="cuda"))
    with pytest.raises(mx.MXFP8Error) as e:
        mx.nvfp4_matvec(D.activations(65, K, seed=3), w)
    assert e.value.status == mx.ERR_UNSUPPORTED
    with pytest.raises(mx.MXFP8Error) as e:
        mx.nvfp4_matvec(x, w, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == mx.ERR_WORKSPACE

    E, H, F = 2, 256, 128
    w1, _ = D.weight(mx, "mxfp8", E * 2 * F, H, seed=1)
    w2, _ = D.weight(mx, "mxfp8", E * H, F, seed=2)
    x = D.activations(2, H, seed=2)
    ids = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    for xs, es, gs in ((x.float(), ids, None), (x, ids.long(), None), (x, ids, torch.ones((2, 2), device="cuda")),
                       (x, ids[:1], None), (x, ids, torch.ones((2, 1), device="cuda").double())):
        with pytest.raises(ValueError):
            mx.moe_decode_fwd(xs, es, gs, *w1, *w2)
    with pytest.raises(ValueError):
        mx.moe_decode_fwd(x, ids, None, w1[0][:256], w1[1], *w2)

    y, r = x, x.clone()
    v = torch.ones(H, device="cuda")
    with pytest.raises(ValueError):
        mx.residual_norm_fwd(y.float(), r)
    with pytest.raises(ValueError):
        mx.residual_norm_fwd(y, r, w_pre=v.bfloat16())
    with pytest.raises(ValueError):
        mx.residual_norm_fwd(y, r, gate=torch.ones((H, 1), device="cuda"))
    with pytest.raises(mx.MXFP8Error):
        mx.residual_norm_fwd(y, r, w_post=v, post_norm=False)


def timeout_child():
    import torch

    import mxfp8_block_scaled_03_gb300 as mx
    E, H, F, T, k = 8, 4096, 2048, 8, 2
    for fmt in ("mxfp8", "nvfp4"):
        w1, _ = D.weight(mx, fmt, E * 2 * F, H, seed=1)
        w2, _ = D.weight(mx, fmt, E * H, F, seed=2)
        x = D.activations(T, H, seed=3)
        ids = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda")
        ws = torch.empty(mx.moe_decode_workspace_size(T, k, H, F, E), dtype=torch.uint8, device="cuda")
        y = D.moe(mx, fmt, x, ids, None, w1, w2, workspace=ws)
        assert mx.mxfp8_check_device_error(ws) == (0, 0)
        os.environ["MXFP8MOE_WAIT_LIMIT_NS"] = "100"
        try:
            D.moe(mx, fmt, x, ids, None, w1, w2, workspace=ws)
            st, bits = mx.mxfp8_check_device_error(ws)
        finally:
            os.environ.pop("MXFP8MOE_WAIT_LIMIT_NS", None)
        assert st == mx.ERR_DEVICE_TIMEOUT and bits & 0x1F00, (st, hex(bits))
        print(f"{fmt}: error bits {bits:#x}", flush=True)
        z = D.moe(mx, fmt, x, ids, None, w1, w2, workspace=ws)
        assert mx.mxfp8_check_device_error(ws) == (0, 0)
        assert torch.equal(y.view(torch.int16), z.view(torch.int16))
    print("ok", flush=True)


def test_waits_that_run_out_are_reported(mx):
    """MXFP8MOE_WAIT_LIMIT_NS shortens the pipeline waits to 100 ns, which a copy from memory cannot meet: the
    call returns, the error word says so, and the next call on the workspace is unharmed (child process)."""
    code = "from tests.test_gpu_decode_edges import timeout_child; timeout_child()"
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr


@FORMATS
@pytest.mark.parametrize("T,K,N", [(1, 4096, 128), (2, 14336, 640), (3, 4352, 1024), (4, 8192, 4096), (1, 2048, 9600),
                                   (9, 4096, 1152), (33, 2048, 384)])
def test_units_shared_by_several_ctas(mx, fmt, T, K, N):
    """Few tiles and long rows: every tile's sum is put together from the parts of several CTAs."""
    w, wv = D.weight(mx, fmt, N, K, seed=T)
    x = D.activations(T, K, seed=K)
    y = D.matvec(mx, fmt, x, w)
    ref, S = x.double() @ wv.t(), D.block_max(x.double(), 32 if fmt == "mxfp8" else 16) @ wv.abs().t()
    D.check(y, ref, 2.0 ** -8 * ref.abs() + 2.0 ** -12 * S + 1e-30)


@FORMATS
@pytest.mark.parametrize("T,k,E,H,F", [(1, 2, 16, 4096, 2048), (2, 3, 4, 2048, 1152), (4, 1, 8, 8192, 384),
                                       (3, 8, 32, 2048, 640)])
def test_experts_shared_by_several_ctas(mx, fmt, T, k, E, H, F):
    w1, v1 = D.weight(mx, fmt, E * 2 * F, H, seed=1)
    w2, v2 = D.weight(mx, fmt, E * H, F, seed=2)
    x = D.activations(T, H, seed=3)
    rng = np.random.default_rng(T)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[0, 0] = -1 if T > 1 else ids[0, 0]      # fewer experts than there may be
    ids, gates = G.to_dev(ids), G.to_dev(rng.random((T, k), dtype=np.float32))
    y = D.moe(mx, fmt, x, ids, gates, w1, w2)
    ref, bound = D.moe_ref(fmt, x, ids, gates, v1, v2, E, H, F)
    D.check(y, ref, bound)
    assert all((D.moe(mx, fmt, x, ids, gates, w1, w2) == y).all() for _ in range(3))


@FORMATS
def test_weights_past_four_gigabytes(mx, fmt):
    """The last expert of a layer of more than 2^32 weight bytes gives, bit for bit, what it gives alone."""
    import torch
    E, H, F = (40, 4096, 14336) if fmt == "mxfp8" else (80, 4096, 14336)
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    gen = torch.Generator(device="cuda").manual_seed(1)

    def rnd(M, K):
        q = torch.randint(0, 120, (M, K if fmt == "mxfp8" else K // 2), dtype=torch.uint8, device="cuda", generator=gen)
        n = mx.mxfp8_sf_bytes(M, K, mx.ROWWISE, mx.SF_MMA) if fmt == "mxfp8" else mx.nvfp4_sf_bytes(M, K, mx.SF_MMA)
        sf = torch.randint(*((110, 118) if fmt == "mxfp8" else (0x20, 0x30)), (n,), dtype=torch.uint8, device="cuda",
                           generator=gen)
        return (q, sf) if fmt == "mxfp8" else (q, sf, torch.full((1,), 0.125, device="cuda"))

    def last(w):   # of E equal shares
        return tuple(t if t.numel() == 1 else t[t.shape[0] // E * (E - 1):] for t in w)
    w1, w2 = rnd(E * 2 * F, H), rnd(E * H, F)
    assert w1[0].numel() > 2 ** 32
    x = D.activations(2, H, seed=2)
    ids, alone = (torch.full((2, 1), e, dtype=torch.int32, device="cuda") for e in (E - 1, 0))
    y = D.moe(mx, fmt, x, ids, None, w1, w2)
    assert torch.isfinite(y.float()).all() and y.any()
    assert torch.equal(y.view(torch.int16), D.moe(mx, fmt, x, alone, None, last(w1), last(w2)).view(torch.int16))


@FORMATS
def test_a_stream_of_its_own(mx, fmt):
    """stream=: the kernels run there, and what the call allocates belongs to that stream."""
    import torch
    w, _ = D.weight(mx, fmt, 256, 512, seed=1)
    x = D.activations(3, 512, seed=2)
    r, v = torch.randn_like(x), torch.ones(512, device="cuda")
    y, (ro, n, st) = D.matvec(mx, fmt, x, w), mx.residual_norm_fwd(x, r, w_pre=v)
    grads = mx.residual_norm_bwd(n, None, x, ro, st, w_pre=v)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                       # the current stream is busy
    z = D.matvec(mx, fmt, x, w, stream=side)
    out = mx.residual_norm_fwd(x, r, w_pre=v, stream=side)
    more = mx.residual_norm_bwd(n, None, x, ro, st, w_pre=v, stream=side)
    side.synchronize()
    assert not torch.cuda.current_stream().query(), "ran on the current stream"
    torch.cuda.synchronize()
    for a, b in zip((y, ro, n, st, *grads), (z, *out, *more)):
        assert (a is None and b is None) or torch.equal(a, b)
