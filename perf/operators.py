"""Cases of the routing and gradient-clipping operators, their plain forms and their values in 64 bits.

A case is one operator at one size:

- ``route``: experts and gates of every token from the router's logits (softmax or sigmoid scores, balance bias,
  expert groups, top-k, renormalised or plain gates), with or without the token-to-expert buckets;
- ``route_backward``: the gradient of the logits from that of the gates and of the balance and z losses;
- ``balance_loss``: the load-balance loss and the z loss of a routing;
- ``grad_norm``, ``grad_clip``: the global norm of a list of gradients, and the list scaled to at most that norm.

The sizes are those of the layers in ``workloads``: d = 64 to 2048, 8 to 1024 experts, up to 131072 tokens.
"""
import math

import torch

own = False

INF = float("inf")


# ---------------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------------
def _route(name, T, N, k, dtype="f32", score="softmax", bias=False, groups=1, top_groups=1, group_score="max",
           renorm=True, scale=1.0, buckets=True, std=1.0, off=0):
    return dict(name=name, op="route", T=T, N=N, k=k, dtype=dtype, score=score, bias=bias, groups=groups,
                top_groups=top_groups, group_score=group_score, renorm=renorm, scale=scale, buckets=buckets, std=std, off=off)


def _backward(name, T, N, k, dtype="f32", score="softmax", renorm=True, scale=1.0, gates=True, balance=0.01, z=0.001,
              std=1.0, off=0):
    return dict(name=name, op="route_backward", T=T, N=N, k=k, dtype=dtype, score=score, renorm=renorm, scale=scale,
                gates=gates, balance=balance, z=z, std=std, off=off)


def _loss(name, T, N, k, dtype="f32", score="softmax", std=1.0, off=0):
    return dict(name=name, op="balance_loss", T=T, N=N, k=k, dtype=dtype, score=score, std=std, off=off)


def _grads(name, op, layers, d, N, dtype="f32", align=1, clip=True):
    return dict(name=name, op=op, layers=layers, d=d, N=N, dtype=dtype, align=align, clip=clip)


def listed():
    return [
        # a decode step of 64 sequences: the experts within the best groups, no buckets
        _route("route_decode", 64, 256, 8, score="sigmoid", bias=True, groups=8, top_groups=4, group_score="top2",
               scale=2.5, buckets=False),
        # the d512_n64 layer's batch, logits of a bf16 router
        _route("route_d512_n64", 4096, 64, 2, dtype="bf16", std=2.2),
        # a training batch of the 256-expert layers with balanced sigmoid routing inside groups
        _route("route_groups", 16384, 256, 8, score="sigmoid", bias=True, groups=8, top_groups=4, group_score="top2",
               scale=2.5),
        # the largest layer's batch, gates as they come out of the softmax
        _route("route_d2048_n1024", 131072, 1024, 4, renorm=False, std=1.4),
        # the d512_n64 training step in bf16
        _backward("backward_d512_n64", 4096, 64, 2, dtype="bf16", std=2.2),
        # sigmoid scores over a number of experts and of tokens that no tile divides
        _backward("backward_sigmoid_odd", 16383, 250, 8, score="sigmoid", scale=2.5, z=0.0),
        # the d1024_n256 training step, gates not renormalised: every logit of a row has a gradient from the gates
        _backward("backward_d1024_n256", 65536, 256, 2, renorm=False),
        # balance loss of the small and of the largest layer
        _loss("balance_d512_n64", 4096, 64, 2, dtype="bf16", std=2.2),
        _loss("balance_d2048_n1024", 131072, 1024, 4, score="sigmoid", std=1.4),
        # one small layer's gradients, packed tightly into one buffer
        _grads("norm_d512_n64", "grad_norm", 1, 512, 64),
        # eight layers of the headline size, a norm above the limit: all is scaled
        _grads("clip_d512_n256", "grad_clip", 8, 512, 256, align=64),
        # 24 layers in bf16, packed tightly
        _grads("clip_d1024_n256", "grad_clip", 24, 1024, 256, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_backward", "balance_loss", "grad_norm", "grad_clip"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("grad_norm", "grad_clip"):
        d = 1 << rng.randint(6, 11)
        N = _log_int(rng, 8, 300)
        per_layer = N * int(math.log2(d)) * d + d * d + N * d
        layers = min(_log_int(rng, 1, 40), max(1, 90_000_000 // per_layer))
        return dict(op=op, layers=layers, d=d, N=N, dtype=dtype, align=rng.choice([1, 8, 64]),
                    clip=rng.random() < 0.7)
    N = _log_int(rng, 8, 1024)
    T = _log_int(rng, 1, min(131072, (1 << 27) // N))
    k = rng.randint(1, 8)
    score = rng.choice(["softmax", "sigmoid"])
    std = rng.uniform(0.5, 3.0)
    off = rng.randint(0, N - k) // 2 if rng.random() < 0.3 else 0
    if op == "balance_loss":
        return dict(op=op, T=T, N=N, k=k, dtype=dtype, score=score, std=std, off=off)
    renorm, scale = rng.random() < 0.6, rng.choice([1.0, 2.5])
    if op == "route_backward":
        what = rng.choice(["gates", "aux", "both"])
        return dict(op=op, T=T, N=N, k=k, dtype=dtype, score=score, renorm=renorm, scale=scale, gates=what != "aux",
                    balance=0.0 if what == "gates" else 0.01, z=0.0 if what == "gates" else rng.choice([0.0, 0.001]),
                    std=std, off=off)
    groups, top_groups = 1, 1
    if rng.random() < 0.5:
        groups = rng.choice([2, 3, 4, 5, 8, 16])
        N = max(groups, N // groups * groups)
        top_groups = rng.randint(1, groups)
        k = min(k, top_groups * (N // groups))
        off = 0
    return dict(op=op, T=T, N=N, k=k, dtype=dtype, score=score, bias=rng.random() < 0.5, groups=groups,
                top_groups=top_groups, group_score=rng.choice(["max", "top2"]), renorm=renorm, scale=scale,
                buckets=rng.random() < 0.7, std=std, off=off)


# ---------------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------------
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _grad_sizes(case):
    """Elements of each gradient of a layer: both sets of angles, the base, its scale, the router and its bias."""
    d, N = case["d"], case["N"]
    angles = N * int(math.log2(d)) * (d // 2)
    return [angles, angles, d * d, 1, N * d, N] * case["layers"]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    st = dict(case=case)
    if case["op"] in ("grad_norm", "grad_clip"):
        # the list is one buffer, each gradient a view of it; out: where the scaled gradients go
        sizes, at, n = _grad_sizes(case), [], 0
        for s in sizes:
            at.append(n)
            n += -(-s // case["align"]) * case["align"]
        flat = (normal(n) * 1e-3).to(_dtype(case))
        out = torch.zeros_like(flat)
        if n > sum(sizes):  # nothing between the gradients
            keep = torch.zeros(n, dtype=torch.bool, device="cuda")
            for o, s in zip(at, sizes):
                keep[o:o + s] = True
            flat = torch.where(keep, flat, torch.zeros_like(flat))
        st.update(flat=flat, out=out, grads=[flat[o:o + s] for o, s in zip(at, sizes)],
                  outs=[out[o:o + s] for o, s in zip(at, sizes)])
        norm = 1e-3 * math.sqrt(sum(sizes))
        st["max_norm"] = 0.37 * norm if case["clip"] else 2.0 * norm
        return st
    T, N, k = case["T"], case["N"], case["k"]
    # logits of normal tokens, each expert with its own offset, as a learned router has them
    logits = (normal(T, N) + math.sqrt(0.5) * normal(N)) * case["std"]
    if case["off"]:  # experts that are switched off
        logits[:, torch.randperm(N, generator=g, device="cuda")[:case["off"]]] = -INF
    st["logits"] = logits.to(_dtype(case))
    if case["op"] == "route":
        st["bias"] = normal(N) * 0.1 if case["bias"] else None
        return st
    # the routing of these logits: k distinct experts a token
    st["idx"] = torch.topk(st["logits"].float(), k, dim=1)[1].to(torch.int32).contiguous()
    if case["op"] == "route_backward":
        st["dgates"] = normal(T, k) if case["gates"] else None
        if case["balance"] or case["z"]:
            load = torch.zeros(N + 1, dtype=torch.int32, device="cuda")
            load[:N] = torch.bincount(st["idx"].reshape(-1).long(), minlength=N).to(torch.int32)
            load[N] = T
            st["load"] = load
            st["dloss"] = torch.tensor([case["balance"], case["z"]], dtype=torch.float32, device="cuda")
        else:
            st["load"] = st["dloss"] = None
    return st


# ---------------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------------
def _unit_softmax(l):
    """exp(l - max) without its sum; masked logits (NaN, -inf) give 0, and +inf ones share the mass."""
    live = l > -INF
    top = torch.where(live, l, -INF).amax(-1, keepdim=True)
    e = torch.where(top == INF, (l == INF).to(l.dtype), torch.exp(l - top))
    return torch.where(live, e, torch.zeros_like(e)), top


def _unit_sigmoid(l):
    """The sigmoid over exp(min(max, 0)) of the row, so that a row of very low logits does not vanish."""
    live = l > -INF
    top = torch.where(live, l, -INF).amax(-1, keepdim=True).clamp(max=0)
    s = torch.where(l > 0, 1 / (1 + torch.exp(-l)), torch.exp(l - top) / (1 + torch.exp(l)))
    return torch.where(live, s, torch.zeros_like(s))


def _over_sum(e):
    total = e.sum(-1, keepdim=True)
    return torch.where(total > 0, e / total, torch.zeros_like(e))


def _scores(l, score):
    live = l > -INF
    if score == "softmax":
        return _over_sum(_unit_softmax(l)[0])
    return torch.where(live, torch.sigmoid(l), torch.zeros_like(l))


def _plain_route(st):
    c = st["case"]
    T, N, k, G = c["T"], c["N"], c["k"], c["groups"]
    l = st["logits"].double()  # which of two near values is larger is decided in 64 bits
    live = l > -INF
    scored = _scores(l, c["score"])
    if st["bias"] is not None:
        scored = scored + st["bias"].double()
    value = l if st["bias"] is None else scored
    live = live & (value > -INF)
    lowest = -1.7e308  # below every value, above what is not a candidate
    value = torch.where(live, value, lowest)
    if G > 1:
        if c["group_score"] == "max":
            of_group = value.view(T, G, N // G).amax(-1)
        else:
            best = torch.where(live, scored, -INF).view(T, G, N // G).topk(min(2, N // G), dim=-1)[0]
            first = best[..., 0]
            of_group = first + torch.where(best[..., -1] > -INF, best[..., -1], 0.0) if N // G > 1 else first
        kept = torch.sort(of_group, dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        value = torch.where(keep.repeat_interleave(N // G, dim=1), value, -INF)
    e = torch.sort(value, dim=1, descending=True, stable=True)[1][:, :k]
    chosen = torch.gather(torch.where(live, l, -INF), 1, e).float()
    if not c["renorm"]:
        gates = torch.gather(torch.where(live, _scores(st["logits"].float(), c["score"]), 0.0), 1, e)
    elif c["score"] == "softmax":
        gates = _over_sum(_unit_softmax(chosen)[0])
    else:
        gates = _over_sum(_unit_sigmoid(chosen))
    gates = gates * c["scale"]
    idx = e.to(torch.int32)
    if not c["buckets"]:
        return idx, gates
    flat = e.reshape(-1)
    counts = torch.bincount(flat, minlength=N)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    rows = torch.sort(flat, stable=True)[1]
    return idx, gates, counts.to(torch.int32), offsets.to(torch.int32), rows.to(torch.int32)


def _plain_backward(st):
    c = st["case"]
    N, k = c["N"], c["k"]
    l = st["logits"].float()
    e = st["idx"].long()
    live = l > -INF
    grad = torch.zeros_like(l)
    if st["dgates"] is not None:
        dg = st["dgates"] * c["scale"]
        chosen = torch.gather(torch.where(live, l, -INF), 1, e)
        if c["score"] == "softmax" and not c["renorm"]:
            p = _scores(l, "softmax")
            pc = torch.gather(p, 1, e)
            grad = -p * (pc * dg).sum(1, keepdim=True)
            grad.scatter_add_(1, e, pc * dg)
        else:
            if c["renorm"]:
                r = _over_sum(_unit_softmax(chosen)[0] if c["score"] == "softmax" else _unit_sigmoid(chosen))
                d = r * (dg - (r * dg).sum(1, keepdim=True))
            else:
                d = dg * _scores(chosen, "sigmoid")
            if c["score"] == "sigmoid":
                d = d * torch.where(chosen > -INF, torch.sigmoid(-chosen), 0.0)
            grad.scatter_add_(1, e, d)
    if st["load"] is not None:
        rows = st["load"][N].float()
        f = st["load"][:N].float() / (k * rows)
        u, top = _unit_softmax(l)
        soft = _over_sum(u)
        p = soft if c["score"] == "softmax" else _over_sum(_unit_sigmoid(l))
        d = p * (f - (p * f).sum(1, keepdim=True)) * (st["dloss"][0] * N / rows)
        if c["score"] == "sigmoid":
            d = d * torch.where(live, torch.sigmoid(-l), 0.0)
        grad = grad + d
        if c["z"]:
            lse = top + torch.log(u.sum(-1, keepdim=True))
            grad = grad + torch.where(live, soft * lse, 0.0) * (2 * st["dloss"][1] / rows)
    return grad.to(st["logits"].dtype)


def _plain_loss(st):
    c = st["case"]
    N, k = c["N"], c["k"]
    l = st["logits"].float()
    some = (l > -INF).any(1)
    u, top = _unit_softmax(l)
    p = _over_sum(u if c["score"] == "softmax" else _unit_sigmoid(l))
    rows = some.sum()
    load = torch.bincount(st["idx"][some].reshape(-1).long(), minlength=N)
    mean = p.double().sum(0) / rows  # long sums
    lse = torch.where(some, (top + torch.log(u.sum(-1, keepdim=True)))[:, 0], 0.0).double()
    loss = torch.stack([N * (load.double() / (k * rows) * mean).sum(), lse.square().sum() / rows]).float()
    return loss, torch.cat([load, rows[None]]).to(torch.int32)


def _plain_norm(st):
    return st["flat"].float().double().square().sum().sqrt()


def _plain_clip(st):
    norm = _plain_norm(st)
    by = torch.where(norm > st["max_norm"], st["max_norm"] / norm, torch.ones_like(norm)).float()
    return norm.float().reshape(1), (st["flat"].float() * by).to(st["flat"].dtype)


# ---------------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------------
def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "route":
        return _plain_route(state)
    if op == "route_backward":
        return _plain_backward(state)
    if op == "balance_loss":
        return _plain_loss(state)
    if op == "grad_norm":
        return _plain_norm(state).float().reshape(1)
    return _plain_clip(state)


def _own(st):
    import ternary_butterfly_experts_b200 as B

    c = st["case"]
    if c["op"] in ("grad_norm", "grad_clip"):
        if "list" not in st:  # kept by a training program as long as its gradients stay where they are
            st["list"] = B.GradList(st["grads"], out=st["outs"] if c["op"] == "grad_clip" else None)
        if c["op"] == "grad_norm":
            return B.bfmoe_grad_norm(st["list"])
        return B.bfmoe_grad_clip(st["list"], st["max_norm"]), st["out"]
    if "ws" not in st:
        st["ws"] = torch.empty(max(256, B.bfmoe_route_workspace_size(c["N"], c["T"], c["k"])), dtype=torch.uint8,
                               device="cuda")
        if c["op"] != "balance_loss":
            st["scoring"] = B.Scoring(score=c["score"], n_groups=c.get("groups", 1),
                                      top_groups=c.get("top_groups", 1), group_score=c.get("group_score", "max"),
                                      renormalize=c["renorm"], scale=c["scale"])
    if c["op"] == "route":
        out = B.bfmoe_route(st["logits"], c["k"], st["scoring"], balance_bias=st["bias"], ws=st["ws"],
                            buckets=c["buckets"])
        return out if c["buckets"] else out[:2]
    if c["op"] == "balance_loss":
        return B.bfmoe_balance_loss(st["logits"], st["idx"], c["score"], ws=st["ws"])
    return B.bfmoe_route_backward(st["logits"], st["idx"], st["scoring"], dgates=st["dgates"], load=st["load"],
                                  dloss=st["dloss"])


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("grad_norm", "grad_clip"):
        n = sum(_grad_sizes(case))
        both = case["op"] == "grad_clip"
        return {"bytes": n * es * (2 if both else 1), "flops": n * (3 if both else 2)}
    T, N, k = case["T"], case["N"], case["k"]
    if case["op"] == "route":
        rest = T * k * 8 + (4 * N if case["bias"] else 0) + ((T * k + 2 * N + 1) * 4 if case["buckets"] else 0)
        return {"bytes": T * N * es + rest, "flops": T * N * (8 + case["k"])}
    if case["op"] == "balance_loss":
        return {"bytes": T * N * es + T * k * 4, "flops": T * N * 8}
    return {"bytes": 2 * T * N * es + T * k * 8, "flops": T * N * 16}


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] not in ("grad_norm", "grad_clip") and case["T"] * case["N"] > 1 << 27:
        return None
    st = prepare(case, seed)
    if case["op"] in ("grad_norm", "grad_clip"):
        x = st["flat"].double()
        norm = torch.linalg.vector_norm(x)
        if case["op"] == "grad_norm":
            return norm.reshape(1)
        return norm.reshape(1), x * min(1.0, st["max_norm"] / float(norm))
    l = st["logits"].double()
    T, N, k = case["T"], case["N"], case["k"]
    lse = torch.logsumexp(l, 1, keepdim=True)
    soft = torch.exp(l - lse)
    s = soft if case["score"] == "softmax" else 0.5 * (1 + torch.tanh(l / 2))
    if case["op"] == "route":
        return _exact_route(case, st, l, s)
    e = st["idx"].long()
    hit = torch.zeros_like(l).scatter_(1, e, 1.0)
    mean = s / s.sum(1, keepdim=True)
    if case["op"] == "balance_loss":
        f = hit.sum(0) / (k * T)
        return torch.stack([N * (f * mean.mean(0)).sum(), (lse ** 2).mean()]), None
    # Jacobians written out: scores by logits, then gates by scores
    grad = torch.zeros_like(l)
    if st["dgates"] is not None:
        ds = torch.zeros_like(l).scatter_(1, e, case["scale"] * st["dgates"].double())
        if case["renorm"]:
            total = (s * hit).sum(1, keepdim=True)
            ds = hit * (ds - (ds * s).sum(1, keepdim=True) / total) / total
        grad += s * (ds - (ds * s).sum(1, keepdim=True)) if case["score"] == "softmax" else ds * s * (1 - s)
    if st["load"] is not None:
        rows = float(st["load"][N])
        dp = float(st["dloss"][0]) * N * st["load"][:N].double() / (k * rows) / rows
        total = s.sum(1, keepdim=True)
        ds = (dp - (dp * mean).sum(1, keepdim=True)) / total
        grad += s * (ds - (ds * s).sum(1, keepdim=True)) if case["score"] == "softmax" else ds * s * (1 - s)
        grad += float(st["dloss"][1]) * 2 / rows * lse * soft
    return grad


def _exact_route(case, st, l, s):
    T, N, k, G = case["T"], case["N"], case["k"], case["groups"]
    with_bias = s if st["bias"] is None else s + st["bias"].double()
    v = (l if st["bias"] is None else with_bias).clone()
    t = torch.arange(T, device=l.device)
    if G > 1:
        per = N // G
        if case["group_score"] == "max":
            of = torch.stack([v[:, g * per:(g + 1) * per].max(1)[0] for g in range(G)], 1)
        else:
            best = [with_bias[:, g * per:(g + 1) * per].sort(1)[0][:, -2:].sum(1) for g in range(G)]
            of = torch.stack(best, 1)
        out = torch.ones(T, N, dtype=torch.bool, device=l.device)
        for _ in range(case["top_groups"]):
            g = of.max(1)[1]
            of[t, g] = -INF
            out &= (torch.arange(N, device=l.device) // per)[None] != g[:, None]
        v[out] = -INF
    picked = []
    for _ in range(k):
        at = v.max(1, keepdim=True)[0]
        # the lowest index among the largest
        e = torch.where(v == at, torch.arange(N, device=l.device)[None], N).min(1)[0]
        picked.append(e)
        v[t, e] = -INF
    e = torch.stack(picked, 1)
    gates = torch.gather(s, 1, e)
    if case["renorm"]:
        gates = gates / gates.sum(1, keepdim=True)
    gates = gates * case["scale"]
    return (e, gates, None, None, None) if case["buckets"] else (e, gates)
