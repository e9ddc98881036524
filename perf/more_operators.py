"""Cases of the operators that close a mixture-of-experts language model's training step, with their plain forms.

Two pairs of operators that meet in the model's objective:
  route   the router's choices from its logits: the k largest, their weights, per-expert counts, the balance loss and
          the loss on the logits' scale; forward and backward;
  lce     the cross entropy of a linear layer over a large vocabulary, without keeping the logits; forward and backward.

The plain forms are elementary torch operations in 32 bits, rounded once at the end.  ``exact`` computes the
definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

MAX_FWD = 4096 * 4096 * 128256          # T * H * V of the largest listed forward
MAX_BWD = 8192 * 4096 * 32000           # and backward
MAX_LOGITS = 32768 * 64                 # T * E of the largest listed router


def listed():
    def route(name, op, T, E, k, dtype, masked=0.0, closed=0.0, normalize=True, spread=False, by_row=False):
        return dict(name=name, op=op, T=T, E=E, k=k, dtype=dtype, masked=masked, closed=closed, normalize=normalize,
                    spread=spread, by_row=by_row)

    def lce(name, op, T, H, V, masked=0.0, zloss=0.0):
        return dict(name=name, op=op, T=T, H=H, V=V, masked=masked, zloss=zloss)

    return [
        # one decode step of a few sequences, many small experts: latency counts
        route("route_fwd_few", "route_fwd", 4, 128, 8, "bf16"),
        # a training batch over few large experts
        route("route_fwd_batch", "route_fwd", 16384, 8, 2, "fp32"),
        # a training batch over many small experts, padded tokens and experts that are closed to some tokens
        route("route_fwd_fine", "route_fwd", 32768, 64, 8, "bf16", masked=0.1, closed=0.3, spread=True),
        # gradients of the two batches; the weights' gradients come in the order of the sorted rows
        route("route_bwd_batch", "route_bwd", 16384, 8, 2, "fp32", by_row=True),
        route("route_bwd_fine", "route_bwd", 32767, 64, 8, "bf16", masked=0.1, closed=0.3, normalize=False),
        # the log-probability of one next token: the weights' bytes
        lce("lce_fwd_token", "lce_fwd", 1, 4096, 32000),
        # a training batch
        lce("lce_fwd_batch", "lce_fwd", 8192, 4096, 32000),
        # half the batch with four times the vocabulary
        lce("lce_fwd_large", "lce_fwd", 4096, 4096, 128256),
        # a ragged, padded batch with an odd vocabulary
        lce("lce_fwd_ragged", "lce_fwd", 1531, 2048, 50257, masked=0.3),
        # a few tokens of a small model: latency, and the weights' and their gradient's bytes
        lce("lce_bwd_few", "lce_bwd", 5, 1024, 32000),
        # the training batch's gradient
        lce("lce_bwd_batch", "lce_bwd", 8192, 4096, 32000),
        # the padded batch's, with a loss on the logits' scale
        lce("lce_bwd_ragged", "lce_bwd", 1531, 2048, 50257, masked=0.3, zloss=1e-3),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route_fwd", "route_bwd", "lce_fwd", "lce_bwd"])
    if op.startswith("route"):
        while True:
            T, E = _log_int(rng, 1, 131072), _log_int(rng, 1, 512)
            if T * E <= MAX_LOGITS:
                break
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, E)), dtype=rng.choice(["bf16", "fp32"]),
                    masked=rng.choice([0.0, 0.2]), closed=rng.choice([0.0, 0.5]), normalize=rng.random() < 0.5,
                    spread=rng.random() < 0.5, by_row=rng.random() < 0.5)
    while True:
        T, H, V = _log_int(rng, 1, 16384), 8 * _log_int(rng, 32, 1024), _log_int(rng, 100, 131072)
        if T * H * V <= (MAX_FWD if op == "lce_fwd" else MAX_BWD):
            break
    return dict(op=op, T=T, H=H, V=V, masked=rng.choice([0.0, 0.4]), zloss=rng.choice([0.0, 1e-3]))


# ---- inputs ---------------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    st = dict(case)
    return (_prepare_route if case["op"].startswith("route") else _prepare_lce)(st, gen)


def _prepare_route(st, gen):
    T, E, k = st["T"], st["E"], st["k"]
    popular = 0.7 * torch.randn(E, generator=gen, device="cuda")
    logits = 1.5 * torch.randn((T, E), generator=gen, device="cuda") + popular
    if st["closed"] > 0:         # experts that a token may not choose; a few tokens may choose none
        closed = torch.rand((T, E), generator=gen, device="cuda") < st["closed"]
        none = torch.rand((T, 1), generator=gen, device="cuda") < 0.01
        logits = logits.masked_fill(closed | none, -math.inf)
    st["mask"] = None
    if st["masked"] > 0:         # padded tokens: whatever is in their logits' place
        st["mask"] = torch.rand(T, generator=gen, device="cuda") >= st["masked"]
        logits = torch.where(st["mask"][:, None], logits, torch.full_like(logits, math.nan))
    st["logits"] = logits.to(torch.bfloat16 if st["dtype"] == "bf16" else torch.float32)
    if st["op"] == "route_fwd":
        if own:
            import mxfp8_block_scaled_03_gb300 as mx
            st["ws"] = torch.empty(mx.moe_route_workspace_size(T, E, k), dtype=torch.uint8, device="cuda")
        return st
    # what the forward left behind, and the incoming gradients
    st["experts"], st["gates"], st["lse"], st["counts"] = _plain_route_fwd(st)[:4]
    st["dgates"] = 0.01 * torch.randn((T, k), generator=gen, device="cuda")
    st["row_of_slot"] = None
    if st["by_row"]:
        st["row_of_slot"] = torch.randperm(T * k, generator=gen, device="cuda").int().view(T, k)
        st["dgates"] = torch.empty_like(st["dgates"]).view(-1).scatter_(0, st["row_of_slot"].view(-1).long(),
                                                                       st["dgates"].view(-1))
    st["dlosses"] = torch.tensor([1e-2, 1e-3], device="cuda")
    return st


def _prepare_lce(st, gen):
    T, H, V = st["T"], st["H"], st["V"]
    w = torch.empty((V, H), dtype=torch.bfloat16, device="cuda")
    for r in range(0, V, 16384):
        n = min(16384, V - r)
        w[r:r + n] = 0.02 * torch.randn((n, H), generator=gen, device="cuda")
    targets = torch.randint(0, V, (T,), generator=gen, device="cuda")
    # normalised activations with a few large channels, leaning towards their target by up to 12 in the logit
    x = torch.randn((T, H), generator=gen, device="cuda")
    big = torch.randint(0, H, (max(1, H // 256),), generator=gen, device="cuda")
    x[:, big] *= 6.0
    wt = w[targets].float()
    x += 12.0 * torch.rand((T, 1), generator=gen, device="cuda") * wt / (wt * wt).sum(-1, keepdim=True)
    if st["masked"] > 0:         # padded or prompt tokens: no target; some of them were never computed
        skip = torch.rand(T, generator=gen, device="cuda") < st["masked"]
        targets = torch.where(skip, torch.full_like(targets, -100), targets)
        if st["op"] == "lce_bwd":
            x = torch.where((skip & (torch.rand(T, generator=gen, device="cuda") < 0.2))[:, None],
                            torch.full_like(x, math.nan), x)
    st["x"], st["w"], st["targets"] = x.bfloat16(), w, targets.int()
    if own:
        import mxfp8_block_scaled_03_gb300 as mx
        size = mx.linear_cross_entropy_workspace_size if st["op"] == "lce_fwd" else \
            mx.linear_cross_entropy_bwd_workspace_size
        st["ws"] = torch.empty(size(T, H, V), dtype=torch.uint8, device="cuda")
    if st["op"] == "lce_fwd":
        return st
    st["lse"] = _plain_lce_fwd(st)[1]
    valid = (st["targets"] >= 0).float()
    n = valid.sum().clamp(min=1)
    st["dloss"] = torch.full((T,), 1.0, device="cuda") / n
    st["dlse"] = (2 * st["zloss"] * st["lse"] / n) if st["zloss"] > 0 else None
    return st


# ---- one pass -------------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    import mxfp8_block_scaled_03_gb300 as mx
    op = st["op"]
    if op == "route_fwd":
        return mx.moe_route_fwd(st["logits"], st["k"], token_mask=st["mask"], normalize=st["normalize"],
                                spread=st["spread"], workspace=st["ws"])
    if op == "route_bwd":
        return mx.moe_route_bwd(st["logits"], st["experts"], st["gates"], st["lse"], st["counts"], dgates=st["dgates"],
                                dlosses=st["dlosses"], row_of_slot=st["row_of_slot"], normalize=st["normalize"])
    if op == "lce_fwd":
        return mx.linear_cross_entropy_fwd(st["x"], st["w"], st["targets"], workspace=st["ws"])
    return mx.linear_cross_entropy_bwd(st["dloss"], st["x"], st["w"], st["targets"], st["lse"], dlse=st["dlse"],
                                       workspace=st["ws"])


def _run_plain(st):
    return {"route_fwd": _plain_route_fwd, "route_bwd": _plain_route_bwd, "lce_fwd": _plain_lce_fwd,
            "lce_bwd": _plain_lce_bwd}[st["op"]](st)


def _plain_route_fwd(st):
    T, E, k, mask = st["T"], st["E"], st["k"], st["mask"]
    l = st["logits"].float()
    if mask is not None:
        l = torch.where(mask[:, None], l, torch.full_like(l, -math.inf))
    top = l.amax(-1, keepdim=True)
    some = top > -math.inf                                   # tokens that take part
    base = torch.where(some, top, torch.zeros_like(top))
    ex = torch.exp(l - base)
    total = ex.sum(-1, keepdim=True)
    lse = (base + torch.log(total)).squeeze(-1)
    p = torch.where(some, ex / total, torch.zeros_like(ex))
    order = torch.sort(l, dim=-1, descending=True, stable=True)
    chosen, ids = order.values[:, :k], order.indices[:, :k]
    real = chosen > -math.inf
    gates = torch.where(real, p.gather(1, ids), torch.zeros_like(chosen))
    if st["normalize"]:
        s = gates.sum(-1, keepdim=True)
        gates = torch.where(s > 0, gates / s, gates)
    counts = torch.zeros(E + 1, dtype=torch.int32, device=l.device)
    counts.index_add_(0, torch.where(real, ids, torch.full_like(ids, E)).view(-1),
                      real.int().view(-1))
    n = some.sum()
    counts[E] = n
    if st["spread"]:
        fill = torch.arange(T * k, device=l.device).view(T, k) % E
    else:
        fill = torch.full_like(ids, -1)
    experts = torch.where(real, ids, fill).int()
    prob_sum = p.sum(0)
    nf = n.float().clamp(min=1)
    balance = (counts[:E].float() * prob_sum).sum() * (E / k) / (nf * nf)
    z = torch.where(some.squeeze(-1), lse * lse, torch.zeros_like(lse)).sum() / nf
    return experts, gates, lse, counts, prob_sum, torch.stack([balance, z])


def _plain_route_bwd(st):
    E, k, ids, gates, lse = st["E"], st["k"], st["experts"].long(), st["gates"], st["lse"]
    some = (lse > -math.inf)[:, None]
    l = torch.where(some, st["logits"].float(), torch.zeros_like(st["logits"].float()))
    p = torch.where(some, torch.exp(l - torch.where(some, lse[:, None], torch.zeros_like(l[:, :1]))),
                    torch.zeros_like(l))
    n = st["counts"][E].float().clamp(min=1)
    c = st["dlosses"][0] * (E / k) * st["counts"][:E].float() / (n * n)
    a = torch.where(some, 2 * st["dlosses"][1] / n * lse[:, None], torch.zeros_like(l[:, :1]))
    d = p * (c - (p * c).sum(-1, keepdim=True) + a)
    dg = st["dgates"] if st["row_of_slot"] is None else st["dgates"][st["row_of_slot"].view(-1).long()].view(ids.shape)
    gd = gates * torch.where(gates > 0, dg, torch.zeros_like(dg))
    s = gd.sum(-1, keepdim=True)
    at = torch.where(gates > 0, ids, torch.zeros_like(ids))
    if st["normalize"]:
        d.scatter_add_(1, at, gd - gates * s)
    else:
        d -= p * s
        d.scatter_add_(1, at, gd)
    return d.to(st["logits"].dtype)


def _plain_lce_fwd(st):
    z = st["x"].float() @ st["w"].float().t()
    top = z.amax(-1, keepdim=True)
    lse = top.squeeze(-1) + torch.log(torch.exp(z - top).sum(-1))
    y = st["targets"].long()
    loss = lse - z.gather(1, y.clamp(min=0)[:, None]).squeeze(-1)
    return torch.where(y >= 0, loss, torch.zeros_like(loss)), lse


def _plain_lce_bwd(st):
    y = st["targets"].long()
    valid = (y >= 0)[:, None]
    x = torch.where(valid, st["x"].float(), torch.zeros((), device="cuda"))
    w = st["w"].float()
    dloss = torch.where(valid, st["dloss"][:, None], torch.zeros((), device="cuda"))
    rate = dloss if st["dlse"] is None else dloss + torch.where(valid, st["dlse"][:, None],
                                                               torch.zeros((), device="cuda"))
    lse = torch.where(valid, st["lse"][:, None], torch.zeros((), device="cuda"))
    dz = torch.exp(x @ w.t() - lse) * rate
    dz.scatter_add_(1, y.clamp(min=0)[:, None], -dloss)
    return (dz @ w).to(st["x"].dtype), (dz.t() @ x).to(st["w"].dtype)


# ---- what a pass cannot do without ----------------------------------------------------------
def work(case):
    op, T = case["op"], case["T"]
    if op.startswith("route"):
        E, k = case["E"], case["k"]
        s = 2 if case["dtype"] == "bf16" else 4
        mask = T if case["masked"] > 0 else 0
        if op == "route_fwd":
            return {"bytes": T * E * s + T * k * 8 + T * 4 + 8 * E + 12 + mask, "flops": 6 * T * E}
        return {"bytes": 2 * T * E * s + T * k * (12 + 4 * case["by_row"]) + T * 4 + 4 * E + 12, "flops": 10 * T * E}
    H, V = case["H"], case["V"]
    if op == "lce_fwd":
        return {"bytes": 2 * H * (T + V) + 12 * T, "flops": 2 * T * H * V}
    n = max(1, round(T * (1.0 - case["masked"])))
    return {"bytes": 4 * H * (T + V) + (16 if case["zloss"] > 0 else 12) * T, "flops": 6 * n * H * V}


# ---- the definitions in 64 bits -------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    return {"route_fwd": _exact_route_fwd, "route_bwd": _exact_route_bwd, "lce_fwd": _exact_lce_fwd,
            "lce_bwd": _exact_lce_bwd}[case["op"]](st)


def _exact_route_fwd(st):
    E, k = st["E"], st["k"]
    l = st["logits"].double()
    if st["mask"] is not None:
        l[~st["mask"]] = -math.inf
    lse = torch.logsumexp(l, -1)
    part = lse > -math.inf
    p = torch.softmax(l, -1)
    p[~part] = 0.0
    gates, p_left, ids = [], l.clone(), torch.arange(E, device="cuda")[None, :]
    counts = torch.zeros(E, dtype=torch.float64, device="cuda")
    for _ in range(k):           # one choice after the other: the largest that is left, the first of equals
        best = p_left.amax(-1, keepdim=True)
        first = torch.where(p_left == best, ids, torch.full_like(ids, E)).amin(-1, keepdim=True)
        here = (ids == first) & (best > -math.inf)
        gates.append((p * here).sum(-1))
        counts += here.sum(0)
        p_left[here] = -math.inf
    gates = torch.stack(gates, 1)
    if st["normalize"]:
        gates = gates / gates.sum(-1, keepdim=True).clamp(min=1e-300)
    n = max(1, int(part.sum()))
    P = p.sum(0)
    balance = E * ((counts / (n * k)) * (P / n)).sum()
    z = (lse[part] ** 2).sum() / n
    return None, gates, lse, None, P, torch.stack([balance, z])


def _exact_route_bwd(st):
    E, k = st["E"], st["k"]
    lse, g, counts = st["lse"].double(), st["gates"].double(), st["counts"].double()
    part = lse > -math.inf
    p = torch.exp(st["logits"].double() - lse[:, None])
    p[~part] = 0.0
    n = max(1.0, float(counts[E]))
    db, dz = (float(v) for v in st["dlosses"])
    e = db * E * counts[:E] / (n * k) / n                    # gradient of each p
    dp = e[None, :].expand_as(p).clone()
    dg = st["dgates"].double()
    if st["row_of_slot"] is not None:
        dg = dg.view(-1)[st["row_of_slot"].long()]
    dg = torch.where(g > 0, dg, torch.zeros_like(dg))
    at = st["experts"].long().clamp(min=0)
    out = torch.zeros_like(p)
    if st["normalize"]:
        out.scatter_add_(1, at, g * (dg - (g * dg).sum(1, keepdim=True)))
    else:
        dp.scatter_add_(1, at, dg)
    out += p * (dp - (p * dp).sum(1, keepdim=True))
    out[part] += p[part] * (2 * dz / n * lse[part])[:, None]
    return out


def _exact_lce_fwd(st):
    x, w, y = st["x"].double(), st["w"], st["targets"].long()
    m = torch.full((st["T"],), -math.inf, dtype=torch.float64, device="cuda")
    s, zy = torch.zeros_like(m), torch.zeros_like(m)
    for v in range(0, st["V"], 8192):                        # a piece of the vocabulary at a time
        z = x @ w[v:v + 8192].double().t()
        new = torch.maximum(m, z.amax(1))
        s = s * torch.exp(m - new) + torch.exp(z - new[:, None]).sum(1)
        m = new
        inside = (y >= v) & (y < v + z.shape[1])
        zy[inside] = z[inside].gather(1, (y[inside] - v)[:, None]).squeeze(1)
    lse = m + torch.log(s)
    return torch.where(y >= 0, lse - zy, torch.zeros_like(lse)), lse


def _exact_lce_bwd(st):
    y = st["targets"].long()
    rows = torch.nonzero(y >= 0).squeeze(1)
    x, t, lse = st["x"][rows].double(), y[rows], st["lse"][rows].double()
    dloss = st["dloss"][rows].double()
    rate = dloss if st["dlse"] is None else dloss + st["dlse"][rows].double()
    dx_rows = torch.zeros_like(x)
    dw = torch.empty(st["w"].shape, dtype=torch.float64, device="cuda")
    for v in range(0, st["V"], 8192):
        w = st["w"][v:v + 8192].double()
        dz = rate[:, None] * torch.exp(x @ w.t() - lse[:, None])
        hit = torch.nonzero((t >= v) & (t < v + len(w))).squeeze(1)
        dz[hit, t[hit] - v] -= dloss[hit]
        dx_rows += dz @ w
        dw[v:v + 8192] = dz.t() @ x
    dx = torch.zeros((st["T"], st["H"]), dtype=torch.float64, device="cuda")
    dx[rows] = dx_rows
    return dx, dw
