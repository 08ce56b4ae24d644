"""Float64 oracle of routing from logits, its gradient, its losses, and the
gradient norm.  TEST INFRASTRUCTURE, like ``bfmoe_oracle``: row by row, from
the definitions, sharing no code with the CUDA path.

Conventions (the pages define expert selection in general only):

* an expert is masked where its logit is NaN or -inf; logits of +inf share
  the whole softmax; the sigmoid of +inf is 1;
* experts rank by logit, or by score + bias when a balance bias is given (a
  NaN or -inf value masks too, without leaving the softmax); lower index first
  on equal values, masked experts last, by index;
* groups of consecutive experts rank by their largest value or the sum of
  their two best scores (+ bias); lower group first; empty groups last;
* gates are the scores of the chosen, 0 for masked ones, over their sum when
  renormalised (0 when nothing is left), times a scale.
"""
from __future__ import annotations

import math

import numpy as np


def live_mask(l: np.ndarray) -> np.ndarray:
    return ~(np.isnan(l) | (l == -np.inf))


def softmax_row(l: np.ndarray) -> np.ndarray:
    live = live_mask(l)
    p = np.zeros(len(l))
    if not live.any():
        return p
    top = l[live].max()
    if top == np.inf:
        p[l == np.inf] = 1.0 / (l == np.inf).sum()
        return p
    p[live] = np.exp(l[live] - top)
    return p / p.sum()


def sigmoid_row(l: np.ndarray) -> np.ndarray:
    s = np.zeros(len(l))
    for e in np.nonzero(live_mask(l))[0]:
        x = float(l[e])
        if x >= 0:
            s[e] = 1.0 / (1.0 + math.exp(-x)) if x < 700 else 1.0
        else:
            s[e] = math.exp(x) / (1.0 + math.exp(x)) if x > -745 else 0.0
    return s


def shares_row(l: np.ndarray, score: str) -> np.ndarray:
    """The scores over their sum.  Sigmoids of very low logits are
    proportional to exp(l): they are divided in that form."""
    if score == "softmax":
        return softmax_row(l)
    live = live_mask(l)
    if not live.any():
        return np.zeros(len(l))
    low = min(float(l[live].max()), 0.0)
    u = np.zeros(len(l))
    for e in np.nonzero(live)[0]:
        x = float(l[e])
        if x > 0:
            u[e] = 1.0 / (1.0 + math.exp(-min(x, 700.0)))
        else:
            u[e] = (math.exp(x - low) if x - low > -745 else 0.0) / (1.0 + (math.exp(x) if x > -745 else 0.0))
    return u / u.sum()


def route_row(l, k, score="softmax", bias=None, groups=1, top_groups=1, group_score="max", renorm=True, scale=1.0):
    """(experts [k], gates [k]) of one row of float64 logits."""
    l = np.asarray(l, np.float64)
    N = len(l)
    live = live_mask(l)
    s = softmax_row(l) if score == "softmax" else sigmoid_row(l)
    with_bias = s if bias is None else s + np.asarray(bias, np.float64)
    value = l.copy() if bias is None else with_bias.copy()
    ranked = live & ~np.isnan(value) & (value != -np.inf)
    value[~ranked] = -np.inf
    per = N // groups
    kept = list(range(groups))
    if top_groups < groups:
        worth = []
        for g in range(groups):
            mine = [e for e in range(g * per, (g + 1) * per) if ranked[e]]
            if not mine:
                worth.append(-np.inf)
            elif group_score == "max":
                worth.append(max(value[e] for e in mine))
            else:
                worth.append(sum(sorted((with_bias[e] for e in mine), reverse=True)[:2]))
        kept = sorted(sorted(range(groups), key=lambda g: (-worth[g], g))[:top_groups])
    cand = [e for g in kept for e in range(g * per, (g + 1) * per)]
    cand.sort(key=lambda e: (not ranked[e], -value[e], e))
    chosen = np.array(cand[:k])
    ok = ranked[chosen]
    if not renorm:
        gates = np.where(ok, s[chosen], 0.0)
    else:
        gates = np.zeros(k)
        if ok.any():
            gates[ok] = shares_row(l[chosen[ok]], score)
    return chosen, gates * scale


def route(logits, k, **kw):
    out = [route_row(l, k, **kw) for l in np.asarray(logits, np.float64)]
    return (np.array([o[0] for o in out], np.int64).reshape(-1, k),
            np.array([o[1] for o in out], np.float64).reshape(-1, k))


def balance_loss(logits, idx, score="softmax"):
    """((balance, z), load [N], rows) over the rows with an expert left."""
    logits = np.asarray(logits, np.float64)
    T, N = logits.shape
    k = idx.shape[1]
    load = np.zeros(N, np.int64)
    P = np.zeros(N)
    z, rows = 0.0, 0
    for t in range(T):
        l = logits[t]
        live = live_mask(l)
        if not live.any():
            continue
        rows += 1
        for e in idx[t]:
            load[e] += 1
        P += shares_row(l, score)
        top = l[live].max()
        lse = top if top == np.inf else top + math.log(np.exp(l[live] - top).sum())
        z += lse * lse
    if rows == 0:
        return (0.0, 0.0), load, 0
    f = load / (k * rows)
    return (N * float((f * P / rows).sum()), z / rows), load, rows


def route_backward_row(l, idx, score="softmax", renorm=True, scale=1.0, dgates=None, load=None, rows=0,
                       dloss=(0.0, 0.0), bias=None):
    """(gradient [N], bound [N]): the gradient of one row, and the sum of the
    magnitudes of the terms it is made of (what rounding errors scale with)."""
    l = np.asarray(l, np.float64)
    N, k = len(l), len(idx)
    live = live_mask(l)
    g, b = np.zeros(N), np.zeros(N)
    if not live.any():
        return g, b
    s = softmax_row(l) if score == "softmax" else sigmoid_row(l)
    one_minus = 1.0 - s if score == "softmax" else np.where(live, sigmoid_row(-np.where(live, l, 0.0)), 0.0)
    if dgates is not None:
        ok = live[idx]
        if bias is not None:
            ok = ok & live_mask(np.asarray(bias, np.float64))[idx]
        dg = np.where(ok, np.asarray(dgates, np.float64), 0.0) * scale
        if score == "softmax" and not renorm:
            pc = np.where(ok, s[idx], 0.0)
            dot, mag = float((pc * dg).sum()), float(np.abs(pc * dg).sum())
            g -= s * dot
            b += s * mag
            for j in range(k):
                g[idx[j]] += pc[j] * dg[j]
                b[idx[j]] += abs(pc[j] * dg[j])
        else:
            r = np.zeros(k)
            if renorm and ok.any():
                r[ok] = shares_row(l[np.asarray(idx)[ok]], score)
            dot, mag = float((r * dg).sum()), float(np.abs(r * dg).sum())
            for j in range(k):
                if not ok[j]:
                    continue
                e = idx[j]
                if renorm:
                    d, m = r[j] * (dg[j] - dot), r[j] * (abs(dg[j]) + mag)
                else:
                    d, m = s[e] * dg[j], s[e] * abs(dg[j])
                f = one_minus[e] if score == "sigmoid" else 1.0
                g[e] += d * f
                b[e] += m * f
    if load is not None and rows > 0:
        f = np.asarray(load[:N], np.float64) / (k * rows)
        p = shares_row(l, score)
        fp = float((f * p).sum())
        c = dloss[0] * N / rows
        w = one_minus if score == "sigmoid" else 1.0
        g += c * p * (f - fp) * w
        b += abs(c) * p * (f + fp) * w
        if dloss[1]:
            top = l[live].max()
            p = softmax_row(l)
            if top == np.inf:  # inf for the experts that share the mass, 0 for the others
                q = np.where(p > 0, np.copysign(np.inf, dloss[1]), 0.0)
            else:
                q = p * (top + math.log(np.exp(l[live] - top).sum())) * 2 * dloss[1] / rows
            g += q
            b += np.abs(q)
    return g, b


def route_backward(logits, idx, dgates=None, **kw):
    out = [route_backward_row(l, idx[t], dgates=None if dgates is None else dgates[t], **kw)
           for t, l in enumerate(np.asarray(logits, np.float64))]
    N = np.asarray(logits).shape[1]
    return (np.array([o[0] for o in out]).reshape(-1, N), np.array([o[1] for o in out]).reshape(-1, N))


def grad_norm(grads) -> float:
    """Square root of the exact sum of squares (math.fsum)."""
    return math.sqrt(math.fsum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads))
