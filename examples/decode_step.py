"""Decoding with the library's operators for a few tokens, and the gradient of the junction around a block.

A stack of blocks runs one step for T sequences.  Per block:

    y        = nvfp4_matvec(o, w_o)                     the attention's output projection (its input o is given)
    r, n     = residual_norm_fwd(y, r, ...)             gate, scaled residual, norm in front of the MoE layer
    logits   = mxfp8_matvec(n, router)
    experts, gates = moe_route_fwd(logits, k)           the k largest, softmax over them
    y        = nvfp4_moe_decode_fwd(n, experts, gates)  the MoE layer
    r, n     = residual_norm_fwd(y, r, ...)             the junction to the next block

The library's calls write to buffers made once, and the step is captured in a CUDA graph and replayed.  It is
checked against the same step in 32-bit PyTorch on the dequantized weights.  The second part trains: the junction as an
autograd function (residual_norm_fwd / residual_norm_bwd) beside the same formula left to autograd.

    python examples/decode_step.py          (on a GB300, after the build, from the repository root)
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp8_block_scaled_03_gb300 as mx  # noqa: E402

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
EPS = 1e-6


def dequantized_nvfp4(w):
    """The values a bf16 matrix has after nvfp4_quantize, in float32 (compact scales, plain torch)."""
    q, sf, amax = mx.nvfp4_quantize(w)
    M, K = w.shape
    table = torch.tensor(E2M1 + [-v for v in E2M1], device=w.device)
    codes = torch.stack((q & 15, q >> 4), dim=-1).view(M, K).long()
    scale = sf.view(torch.float8_e4m3fn).float().view(M, K // 16) * (amax / (6.0 * 448.0))
    return table[codes] * scale.repeat_interleave(16, dim=1)


def dequantized_mxfp8(w):
    q, sf, _, _ = mx.mxfp8_quantize(w)
    scale = torch.exp2(sf.float() - 127.0).view(w.shape[0], -1)
    return q.view(torch.float8_e4m3fn).float() * scale.repeat_interleave(32, dim=1)


class Block:
    """Weights of one block: quantized for the library, and their values for the plain step."""

    def __init__(self, H, F, E, k, device):
        self.H, self.F, self.E, self.k = H, F, E, k

        def rnd(m, n):
            return (0.02 * torch.randn(m, n, device=device)).bfloat16()
        w_o, router, w1, w2 = rnd(H, H), rnd(E, H), rnd(E * 2 * F, H), rnd(E * H, F)
        self.w_o = mx.nvfp4_quantize(w_o, sf_layout=mx.SF_MMA)
        self.router = mx.mxfp8_quantize(router, sf_layout=mx.SF_MMA)[:2]
        self.w1 = mx.nvfp4_quantize(w1, sf_layout=mx.SF_MMA)
        self.w2 = mx.nvfp4_quantize(w2, sf_layout=mx.SF_MMA)
        self.plain = dequantized_nvfp4(w_o), dequantized_mxfp8(router), dequantized_nvfp4(w1), dequantized_nvfp4(w2)
        self.norms = [1.0 + 0.1 * torch.randn(H, device=device) for _ in range(4)]   # post, pre; twice
        self.gate = 0.5 + torch.rand(H, device=device)


class Decoder:
    """Blocks, and what a step of T sequences writes: allocated once."""

    def __init__(self, blocks, T, res_scale=0.9):
        H, F, E, k = blocks[0].H, blocks[0].F, blocks[0].E, blocks[0].k
        device = blocks[0].gate.device
        self.blocks, self.T, self.res_scale = blocks, T, res_scale
        self.r = torch.empty((T, H), device=device)                       # residual stream, 32 bits
        self.n, self.y = (torch.empty((T, H), dtype=torch.bfloat16, device=device) for _ in range(2))
        self.o = torch.empty((len(blocks), T, H), dtype=torch.bfloat16, device=device)
        self.stats = torch.empty((2, T), device=device)
        self.logits = torch.empty((T, E), dtype=torch.bfloat16, device=device)
        self.linear_ws = torch.empty(mx.matvec_workspace_size(T, H), dtype=torch.uint8, device=device)
        self.moe_ws = torch.empty(mx.moe_decode_workspace_size(T, k, H, F, E), dtype=torch.uint8, device=device)
        self.choices = [torch.empty((T, k), dtype=torch.int32, device=device) for _ in blocks]
        # what moe_route_fwd writes beside the choices: weights, lse, counts, sums of the probabilities, losses
        self.routed = (torch.empty((T, k), device=device), torch.empty(T, device=device),
                       torch.empty(E + 1, dtype=torch.int32, device=device), torch.empty(E, device=device),
                       torch.empty(2, device=device))
        self.route_ws = torch.empty(max(16, mx.moe_route_workspace_size(T, E, k)), dtype=torch.uint8, device=device)

    def step(self):
        out = (self.r, self.n, self.stats)
        for b, o, choices in zip(self.blocks, self.o, self.choices):
            mx.nvfp4_matvec(o, b.w_o, out=self.y, workspace=self.linear_ws)
            mx.residual_norm_fwd(self.y, self.r, w_post=b.norms[0], w_pre=b.norms[1], res_scale=self.res_scale,
                                 eps=EPS, out=out)
            mx.mxfp8_matvec(self.n, *b.router, out=self.logits, workspace=self.linear_ws)
            mx.moe_route_fwd(self.logits, b.k, out=(choices, *self.routed), workspace=self.route_ws)
            mx.nvfp4_moe_decode_fwd(self.n, choices, self.routed[0], b.w1, b.w2, out=self.y, workspace=self.moe_ws)
            mx.residual_norm_fwd(self.y, self.r, w_post=b.norms[2], gate=b.gate, w_pre=b.norms[3],
                                 res_scale=self.res_scale, eps=EPS, out=out)

    def plain_step(self, r):
        """The same step in float32 on the dequantized weights, with the choices the step made."""
        def rms(v):
            return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
        for b, o, choices in zip(self.blocks, self.o, self.choices):
            w_o, router, w1, w2 = b.plain
            r = self.res_scale * r + rms(o.float() @ w_o.t()) * b.norms[0]
            n = rms(r) * b.norms[1]
            gates = torch.softmax((n @ router.t()).gather(1, choices.long()), dim=-1)
            w1, w2 = w1.view(b.E, 2 * b.F, b.H), w2.view(b.E, b.H, b.F)
            y = torch.zeros_like(r)
            for t in range(self.T):
                for j in range(b.k):
                    e = choices[t, j]
                    gu = w1[e] @ n[t]
                    y[t] += gates[t, j] * (w2[e] @ (torch.nn.functional.silu(gu[:b.F]) * gu[b.F:]))
            r = self.res_scale * r + b.gate * rms(y) * b.norms[2]
        return r


class ResidualNorm(torch.autograd.Function):
    """(res_out, n) of residual_norm_fwd with the gradients of residual_norm_bwd."""

    @staticmethod
    def forward(ctx, y, res, w_post, gate, w_pre, res_scale):
        res_out, n, stats = mx.residual_norm_fwd(y, res, w_post, gate, w_pre, res_scale=res_scale, eps=EPS)
        ctx.save_for_backward(y, res_out, stats, w_post, gate, w_pre)
        ctx.res_scale = res_scale
        return res_out, n

    @staticmethod
    def backward(ctx, dres_out, dn):
        y, res_out, stats, w_post, gate, w_pre = ctx.saved_tensors
        return (*mx.residual_norm_bwd(dn.contiguous(), dres_out.contiguous(), y, res_out, stats, w_post, gate, w_pre,
                                      res_scale=ctx.res_scale), None)


def decode(T=4, layers=4, H=1024, F=512, E=128, k=8):
    """Runs and checks a step; returns (error relative to the result's norm, us per replayed step)."""
    dec = Decoder([Block(H, F, E, k, "cuda") for _ in range(layers)], T)
    r0 = torch.randn(T, H, device="cuda")
    dec.o.normal_()
    dec.r.copy_(r0)
    dec.step()
    ref = dec.plain_step(r0)
    err = float((dec.r - ref).norm() / ref.norm())
    first = dec.r.clone()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        dec.step()
    dec.r.copy_(r0)
    graph.replay()
    assert torch.equal(dec.r, first), "a replayed step differs from a direct one"
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    t0.record()
    for _ in range(20):
        graph.replay()
    t1.record()
    torch.cuda.synchronize()
    assert mx.mxfp8_check_device_error(dec.moe_ws)[0] == mx.OK
    return err, t0.elapsed_time(t1) * 1e3 / 20


def train(T=512, H=1024):
    """Gradients through ResidualNorm against autograd on the formula; returns the largest relative error."""
    def leaf(*shape, dtype=torch.float32):
        return torch.randn(*shape, device="cuda").to(dtype).requires_grad_()
    y, res = leaf(T, H, dtype=torch.bfloat16), leaf(T, H)
    w_post, gate, w_pre = leaf(H), leaf(T, 1), leaf(H)
    inputs = (y, res, w_post, gate, w_pre)
    a, b = torch.randn(T, H, device="cuda"), torch.randn(T, H, device="cuda").bfloat16()
    res_out, n = ResidualNorm.apply(*inputs, 0.9)
    got = torch.autograd.grad(((res_out * a).sum() + (n * b).sum().float()), inputs)

    def rms(v):
        return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    plain = 0.9 * res + gate * (rms(y.float()) * w_post)
    want = torch.autograd.grad((plain * a).sum() + (rms(plain) * w_pre * b.float()).sum(), inputs)
    return max(float((g.float() - w.float()).norm() / w.float().norm()) for g, w in zip(got, want))


if __name__ == "__main__":
    torch.manual_seed(0)
    err, us = decode()
    print(f"decode: error {err:.2e}, {us:.1f} us a step of 4 blocks")
    grad_err = train()
    print(f"train: error of the gradients {grad_err:.2e}")
    # bf16 roundings of y, n and the logits (2^-9 each), a handful of them per block
    assert err < 0.02 and grad_err < 0.01
