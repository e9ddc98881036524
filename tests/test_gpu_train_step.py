"""The router, the MoE layer, the junction and the cross entropy run together, forward and backward."""
import os
import subprocess
import sys

import pytest

from tests import test_gpu_decode as D

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

mx = D.mx


def test_train_step_example(mx):
    r = subprocess.run([sys.executable, os.path.join("examples", "train_step.py")], cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "gradients: worst" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("spread", [True, False])
def test_routed_layer_with_masked_tokens(mx, spread):
    """Masked tokens through either form of the layer: spread slots through the grouped calls, dropped ones through the
    decode call.  Both give zeros for masked tokens and agree for the others (activations in 8 bits against bf16: each
    rounding to E4M3 is off by at most 2^-4, four of them in the layer, independent over 128 and more products)."""
    import torch
    torch.manual_seed(1)
    T, E, H, F, k = 40, 8, 256, 384, 2
    x = torch.randn(T, H, device="cuda").bfloat16()
    w1 = (0.05 * torch.randn(E * 2 * F, H, device="cuda")).bfloat16()
    w2 = (0.05 * torch.randn(E * H, F, device="cuda")).bfloat16()
    w1q, w2q = (mx.mxfp8_quantize(w, sf_layout=mx.SF_MMA)[:2] for w in (w1, w2))
    mask = torch.rand(T, device="cuda") < 0.7
    logits = torch.randn(T, E, device="cuda")
    logits[~mask] = float("nan")
    experts, gates, _, counts, _, _ = mx.moe_route_fwd(logits, k, token_mask=mask, spread=spread)
    if spread:
        split, row_of_slot, token_of_row, gates_sorted, ws = mx.moe_permute(experts, gates, E)
        assert mx.mxfp8_check_device_error(ws) == (0, 0)
        assert int(split.sum()) == T * k and int(counts[:E].sum()) == k * int(mask.sum())
        out = mx.moe_combine(mx.grouped_mlp_fwd_tokens(x, token_of_row, split, gates_sorted, *w1q, *w2q), row_of_slot)
    else:
        assert (experts[~mask] == -1).all()
        out = mx.moe_decode_fwd(x, experts, gates, *w1q, *w2q)
    assert not out[~mask].any()
    plain, _, _, _, _, _ = mx.moe_route_fwd(torch.where(mask[:, None], logits, 0.0), k)
    g = torch.where(mask[:, None], gates, 0.0)
    ref = mx.moe_decode_fwd(x, plain, g, *w1q, *w2q)
    err = (out[mask].float() - ref[mask].float()).norm() / ref[mask].float().norm()
    assert err <= (4 * 2.0 ** -4 if spread else 0.0)
