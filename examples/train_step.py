"""A training step of a small mixture-of-experts language model with the library's operators, as autograd functions.

    e        = embedding[tokens]
    logits   = e @ router                               (torch)
    route    = moe_route_fwd(logits, token_mask)        choices, weights, counts, balance loss and loss on lse
    y        = moe_permute, grouped_mlp_fwd_tokens_train, moe_combine           the MoE layer, in MXFP8
    r, n     = residual_norm_fwd(y, e, ...)             the scaled residual and the norm in front of the head
    loss     = linear_cross_entropy_fwd(n, head, targets)                       without the logits over the vocabulary

The backward runs linear_cross_entropy_bwd, residual_norm_bwd, grouped_mlp_bwd_tokens and moe_route_bwd, which takes
the routing weights' gradients in the order of the sorted rows, as the one before it writes them.  Padded tokens have no
target and are masked in the router.  The gradients are checked against the same step with the router and the cross entropy
left to autograd in 32 bits; then a few steps of plain gradient descent follow.

    python examples/train_step.py          (on a GB300, after the build, from the repository root)
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp8_block_scaled_03_gb300 as mx  # noqa: E402

EPS = 1e-6


class Experts:
    """The experts' weights, quantized along both axes (rows for the forward, columns for the backward)."""

    def __init__(self, E, H, F, device):
        self.E, self.H, self.F = E, H, F
        w1 = (0.05 * torch.randn(E * 2 * F, H, device=device)).bfloat16()
        w2 = (0.05 * torch.randn(E * H, F, device=device)).bfloat16()
        self.w1, self.w2 = (mx.mxfp8_quantize(w, sf_layout=mx.SF_MMA)[:2] for w in (w1, w2))
        self.w1t, self.w2t = mx.mxfp8_quantize_colwise_t(w1), mx.mxfp8_quantize_colwise_t(w2)


class Route(torch.autograd.Function):
    """(losses, experts, gates, gates of the sorted rows, and the permutation) from the router's logits.  The gates'
    gradient arrives in the sorted rows' order."""

    @staticmethod
    def forward(ctx, logits, k, mask):
        experts, gates, lse, counts, _, losses = mx.moe_route_fwd(logits, k, token_mask=mask, spread=True)
        split, row_of_slot, token_of_row, gates_sorted, _ = mx.moe_permute(experts, gates, logits.shape[1])
        ctx.save_for_backward(logits, experts, gates, lse, counts, row_of_slot)
        ctx.mark_non_differentiable(experts, split, row_of_slot, token_of_row, gates, counts)
        return losses, gates_sorted, experts, gates, split, row_of_slot, token_of_row, counts

    @staticmethod
    def backward(ctx, dlosses, dgates_sorted, *_):
        logits, experts, gates, lse, counts, row_of_slot = ctx.saved_tensors
        return mx.moe_route_bwd(logits, experts, gates, lse, counts, dgates=dgates_sorted.contiguous(),
                                dlosses=dlosses.contiguous(), row_of_slot=row_of_slot), None, None


class MoE(torch.autograd.Function):
    """The MoE layer on the sorted rows; x and the gates get gradients (the experts stay as they are here)."""

    @staticmethod
    def forward(ctx, x, gates_sorted, split, row_of_slot, token_of_row, w):
        rows, saved = mx.grouped_mlp_fwd_tokens_train(x, token_of_row, split, gates_sorted, *w.w1, *w.w2)
        ctx.save_for_backward(x, gates_sorted, split, row_of_slot, token_of_row, saved)
        ctx.w = w
        return mx.moe_combine(rows, row_of_slot)

    @staticmethod
    def backward(ctx, dy):
        x, gates_sorted, split, row_of_slot, token_of_row, saved = ctx.saved_tensors
        w = ctx.w
        dx_rows, dgates, _, _, _ = mx.grouped_mlp_bwd_tokens(x, token_of_row, split, gates_sorted, saved, *w.w1t, *w.w2t,
                                                             dy.contiguous())
        return mx.moe_combine(dx_rows, row_of_slot), dgates, None, None, None, None


class ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, res, w_pre):
        res_out, n, stats = mx.residual_norm_fwd(y, res, w_pre=w_pre, post_norm=False, eps=EPS)
        ctx.save_for_backward(y, res_out, stats, w_pre)
        return res_out, n

    @staticmethod
    def backward(ctx, dres_out, dn):
        y, res_out, stats, w_pre = ctx.saved_tensors
        dy, dres, _, _, dw = mx.residual_norm_bwd(dn.contiguous(), dres_out.contiguous(), y, res_out, stats, w_pre=w_pre,
                                                  post_norm=False)
        return dy, dres, dw


class LinearCrossEntropy(torch.autograd.Function):
    """(loss, lse) per token; negative targets take no part."""

    @staticmethod
    def forward(ctx, x, w, targets):
        loss, lse = mx.linear_cross_entropy_fwd(x, w, targets)
        ctx.save_for_backward(x, w, targets, lse)
        return loss, lse

    @staticmethod
    def backward(ctx, dloss, dlse):
        x, w, targets, lse = ctx.saved_tensors
        dx, dw = mx.linear_cross_entropy_bwd(dloss.contiguous(), x, w, targets, lse, dlse=dlse.contiguous())
        return dx, dw, None


class Model:
    def __init__(self, V, H, F, E, k, device="cuda"):
        self.k, self.experts = k, Experts(E, H, F, device)

        def leaf(scale, *shape, dtype=torch.float32):
            return (scale * torch.randn(*shape, device=device)).to(dtype).requires_grad_()
        self.embedding = leaf(1.0, V, H, dtype=torch.bfloat16)
        self.router = leaf(0.1, H, E)
        self.norm = torch.ones(H, device=device, requires_grad=True)
        self.head = leaf(0.02, V, H, dtype=torch.bfloat16)
        self.leaves = (self.embedding, self.router, self.norm, self.head)

    def objective(self, tokens, targets, plain=False):
        """(objective, mean cross entropy, counts): cross entropy, 1e-2 times the balance loss, 1e-3 times the mean squared
        lse of the router, 1e-4 times that of the head."""
        mask = targets >= 0
        e = self.embedding[tokens]
        logits = e.float() @ self.router
        # the choices come from the operator either way; plain: their weights and the losses from autograd
        losses, gates_sorted, experts, gates, split, row_of_slot, token_of_row, counts = Route.apply(logits, self.k, mask)
        if plain:
            losses, gates_sorted = self.plain_route(logits, mask, experts, gates, row_of_slot, counts)
        y = MoE.apply(e, gates_sorted, split, row_of_slot, token_of_row, self.experts)
        _, n = ResidualNorm.apply(y, e, self.norm)
        if plain:
            z = n.float() @ self.head.float().t()
            lse = torch.logsumexp(z, -1)
            loss = torch.where(mask, lse - z.gather(1, targets.clamp(min=0)[:, None])[:, 0], 0.0)
        else:
            loss, lse = LinearCrossEntropy.apply(n, self.head, targets)
        count = mask.sum().clamp(min=1)
        ce = loss.sum() / count
        # lse of rows without a target exists, but takes no part
        return ce + 1e-2 * losses[0] + 1e-3 * losses[1] + 1e-4 * torch.where(mask, lse * lse, 0.0).sum() / count, ce, counts

    def plain_route(self, logits, mask, experts, gates, row_of_slot, counts):
        E = logits.shape[1]
        l = logits.masked_fill(~mask[:, None], 0.0)
        lse, p = torch.logsumexp(l, -1), torch.softmax(l, -1)
        g = p.gather(1, experts.long())
        g = torch.where(mask[:, None], g / g.sum(-1, keepdim=True), 0.0)
        n = counts[E].float()
        f = counts[:E].float() / (n * self.k)
        balance = E * (f * (p * mask[:, None]).sum(0) / n).sum()
        sorted_gates = torch.zeros(gates.numel(), device=g.device).scatter(0, row_of_slot.view(-1).long(), g.view(-1))
        return torch.stack([balance, (lse * lse * mask).sum() / n]), sorted_gates


def run(T=512, V=5000, H=256, F=512, E=8, k=2, steps=3):
    """Largest relative difference of a leaf's gradient to the plain step's, and the cross entropy before and after."""
    model = Model(V, H, F, E, k)
    tokens = torch.randint(0, V, (T,), device="cuda")
    targets = torch.randint(0, V, (T,), device="cuda")
    targets[-T // 5:] = -1                                    # padding
    got = torch.autograd.grad(model.objective(tokens, targets)[0], model.leaves)
    want = torch.autograd.grad(model.objective(tokens, targets, plain=True)[0], model.leaves)
    worst = max(float((g.float() - w.float()).norm() / w.float().norm()) for g, w in zip(got, want))
    first = last = None
    for _ in range(steps):
        objective, ce, counts = model.objective(tokens, targets)
        assert int(counts[:E].sum()) == k * int(counts[E]) == k * int((targets >= 0).sum())
        grads = torch.autograd.grad(objective, model.leaves)
        assert all(bool(torch.isfinite(g).all()) for g in grads)
        with torch.no_grad():
            for leaf, g in zip(model.leaves, grads):
                leaf -= 0.5 * g
        first, last = float(ce.detach()) if first is None else first, float(ce.detach())
    return worst, first, last


if __name__ == "__main__":
    torch.manual_seed(0)
    worst, first, last = run()
    print(f"gradients: worst relative difference to the plain step {worst:.2e}; cross entropy {first:.3f} -> {last:.3f}")
    # the roundings of dz, dx and dw to bf16 (2^-8 each), and those behind them in the MXFP8 layer's gradient
    assert worst < 0.03
