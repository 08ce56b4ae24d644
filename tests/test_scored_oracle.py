"""The routing oracle (oracle/scored_oracle.py) against worked examples, the
plain top-k oracle and finite differences."""
import math

import numpy as np
import pytest

from oracle import bfmoe_oracle as O
from oracle import scored_oracle as S


def test_plain_softmax_is_the_plain_router():
    rng = np.random.default_rng(0)
    l = rng.normal(size=(50, 12))
    idx, gates = S.route(l, 3)
    ref, _ = O.topk(l, 3)
    assert np.array_equal(idx, ref)
    assert np.allclose(gates, O.gates_for(l, ref), rtol=1e-14)


def test_worked_sigmoid_groups():
    # sigmoid scores 0.5 0.8 | 0.9 0.1 | 0.6 0.7 with a bias on expert 0
    logit = lambda p: math.log(p / (1 - p))  # noqa: E731
    l = np.array([logit(p) for p in (0.5, 0.8, 0.9, 0.1, 0.6, 0.7)])
    kw = dict(score="sigmoid", groups=3, renorm=True, scale=2.0)
    bias = np.array([0.25, 0, 0, 0, 0, 0.0])         # group sums 1.55, 1.0, 1.3
    idx, g = S.route_row(l, 2, bias=bias, top_groups=2, group_score="top2", **kw)
    assert list(idx) == [1, 0]                       # 0.8, then 0.5 + 0.25 (0.9 is not in a kept group)
    assert np.allclose(g, [2 * 0.8 / 1.3, 2 * 0.5 / 1.3])
    idx, g = S.route_row(l, 2, top_groups=1, group_score="max", **kw)
    assert list(idx) == [2, 3] and np.allclose(g, [1.8, 0.2])


def test_masks_and_infinities():
    ninf, inf, nan = -np.inf, np.inf, np.nan
    idx, g = S.route_row([ninf, 1.0, nan, ninf], 3)
    assert list(idx) == [1, 0, 2] and list(g) == [1, 0, 0]
    idx, g = S.route_row([ninf] * 4, 2, score="sigmoid")
    assert list(idx) == [0, 1] and list(g) == [0, 0]
    idx, g = S.route_row([0.0, inf, 3.0, inf], 3)
    assert list(idx) == [1, 3, 2] and np.allclose(g, [0.5, 0.5, 0])
    low = float(np.finfo(np.float32).min)
    idx, g = S.route_row([low, low, low], 2, score="sigmoid")
    assert list(idx) == [0, 1] and np.allclose(g, 0.5)
    idx, g = S.route_row([1.0, 2.0, 3.0], 2, bias=[0.0, ninf, 0.0])
    assert list(idx) == [2, 0] and g[0] > g[1] > 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gate_gradient_by_differences(score, renorm):
    rng = np.random.default_rng(5)
    N, k = 9, 3
    l = rng.normal(size=N) * 1.5
    l[4] = -np.inf
    dg = rng.normal(size=k)
    kw = dict(score=score, renorm=renorm, scale=1.7)
    idx, _ = S.route_row(l, k, **kw)
    g, bound = S.route_backward_row(l, idx, dgates=dg, **kw)
    assert (np.abs(g) <= bound + 1e-15).all() and g[4] == 0
    for e in range(N):
        if e == 4:
            continue
        h = 1e-6
        lp, lm = l.copy(), l.copy()
        lp[e] += h
        lm[e] -= h
        (ip, gp), (im, gm) = S.route_row(lp, k, **kw), S.route_row(lm, k, **kw)
        assert np.array_equal(ip, idx) and np.array_equal(im, idx)
        num = float(((gp - gm) * dg).sum()) / (2 * h)
        assert abs(num - g[e]) < 1e-8


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_loss_gradient_by_differences(score):
    rng = np.random.default_rng(6)
    T, N, k = 5, 7, 2
    l = rng.normal(size=(T, N)) * 1.3
    l[2] = -np.inf                      # an empty row counts nowhere
    l[3, 1] = np.nan
    idx, _ = S.route(l, k, score=score)
    (bal, z), load, rows = S.balance_loss(l, idx, score)
    assert rows == T - 1 and load.sum() == k * rows
    g, _ = S.route_backward(l, idx, score=score, load=load, rows=rows, dloss=(0.3, 0.7))
    assert (g[2] == 0).all() and g[3, 1] == 0
    for t in range(T):
        for e in range(N):
            if not np.isfinite(l[t, e]):
                continue
            h = 1e-6
            out = []
            for s in (h, -h):
                m = l.copy()
                m[t, e] += s
                (b2, z2), _, _ = S.balance_loss(m, idx, score)
                out.append(0.3 * b2 + 0.7 * z2)
            assert abs((out[0] - out[1]) / (2 * h) - g[t, e]) < 1e-8


def test_balanced_routing_has_loss_one():
    l = np.zeros((8, 4))
    idx = np.array([[t % 4] for t in range(8)])
    (bal, z), load, rows = S.balance_loss(l, idx)
    assert abs(bal - 1.0) < 1e-14 and abs(z - math.log(4) ** 2) < 1e-14


def test_grad_norm_is_the_norm_of_all():
    rng = np.random.default_rng(1)
    gs = [rng.normal(size=s) for s in ((3, 4), (1,), (0,), (17,))]
    assert abs(S.grad_norm(gs) - np.linalg.norm(np.concatenate([g.ravel() for g in gs]))) < 1e-14
