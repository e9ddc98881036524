"""A CTA's shared memory may be touched by its cluster only once that CTA is known to run: in every kernel of the router
(and of the cross entropy) a cluster barrier stands before the first access to another CTA's shared memory.  Read from the
source, because a CTA that comes too early can fault the GPU; the GPU test runs the kernel where CTAs without experts come
to that access at once."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp8_block_scaled_03_gb300", "csrc")
REMOTE = re.compile(r"st_remote_u32\(|load_remote\(|mbar_arrive_remote\(|tma_load_2d_pair\(|tc_commit_pair_both\(")


@pytest.mark.parametrize("name", ["moe_route.cu", "cross_entropy.cu"])
def test_a_barrier_stands_before_the_first_remote_access(name):
    with open(os.path.join(CSRC, name)) as f:
        source = re.sub(r"//[^\n]*", "", f.read())
    kernels = re.split(r"\n__global__ ", source)[1:]
    seen = 0
    for k in kernels:
        body = k[:k.index("\n}\n")]
        first = REMOTE.search(body)
        if first is not None:
            seen += 1
            assert 0 <= body.find("cluster_sync_all()") < first.start(), body[:80]
    assert seen == {"moe_route.cu": 2, "cross_entropy.cu": 1}[name]


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,dtype", [(40000, 1, 1, "fp32"), (33000, 3, 2, "bf16"), (70000, 4, 4, "fp32"), (20000, 7, 2, "bf16"),
                                         (20000, 9, 3, "fp32")])
def test_fewer_experts_than_ctas_that_join_their_sums(T, E, k, dtype):
    """More than 64 passes, so that a second kernel joins the sums, with CTAs that have no expert.  Whole numbers are equal;
    prob_sum is off by 512 terms in sequence and a tree (2^-14), balance by that and its own sum."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import mxfp8_block_scaled_03_gb300 as mx
    gen = torch.Generator(device="cuda").manual_seed(E)
    logits = torch.randn((T, E), generator=gen, device="cuda").to(torch.float32 if dtype == "fp32" else torch.bfloat16)
    p = torch.softmax(logits.double(), 1)
    lse = torch.logsumexp(logits.double(), 1)
    first = None
    for _ in range(50):
        experts, _, _, counts, prob_sum, losses = mx.moe_route_fwd(logits, k)
        if first is None:
            first = counts, prob_sum, losses
            want = torch.bincount(experts.view(-1).long(), minlength=E)
            assert torch.equal(counts[:E].long(), want) and int(counts[E]) == T
            P = p.sum(0)
            assert ((prob_sum.double() - P).abs() <= 2.0 ** -14 * P).all()
            both = torch.stack([E * (want.double() * P).sum() / (float(T) ** 2 * k), (lse * lse).mean()])
            assert ((losses.double() - both).abs() <= 2.0 ** -13 * both).all()
        assert all(torch.equal(a, b) for a, b in zip(first, (counts, prob_sum, losses)))
