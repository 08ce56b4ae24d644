"""The operators together, as a training step and a serving step use them:
logits, routing, experts, losses, gradients of experts, gates and logits, the
clipped list; against the float64 oracles."""
import os

import numpy as np
import pytest

import workloads as W
from oracle import bfmoe_oracle as O
from oracle import scored_oracle as S

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import ternary_butterfly_experts_b200.build as b
    b.build()


def B():
    import ternary_butterfly_experts_b200 as m
    return m


def setup(d, N, k, T, dtype, seed):
    wl = W.custom("scored", d=d, n_experts=N, k=k, tokens=T, dtype=dtype, bias_var=0.5)
    inp = W.generate(wl, seed=seed)
    layer = B().Layer.from_host(inp.w_base, inp.alpha, inp.theta, inp.phi)
    return inp, layer, inp.x.cuda().contiguous(), torch.from_numpy(inp.w_gate).cuda(), torch.from_numpy(inp.bias).cuda()


@pytest.mark.parametrize("d,N,T,dtype", [(64, 8, 33, "f32"), (64, 40, 130, "bf16"), (512, 256, 257, "bf16"),
                                         (32, 12, 50, "bf16"), (128, 33, 1, "bf16"), (256, 1, 9, "f32"),
                                         (1024, 100, 129, "bf16")])
def test_router_logits(d, N, T, dtype):
    inp, _, x, wg, bias = setup(d, N, min(2, N), T, dtype, d + N)
    for b in (bias, None):
        got = B().bfmoe_router_logits(x, wg, b).cpu().numpy()
        ref = O.router_logits(inp.x_f64(), inp.w_gate, inp.bias if b is not None else None)
        # a float32 sum of d products: d half steps of the sum of magnitudes at worst
        mag = np.abs(inp.x_f64()) @ np.abs(inp.w_gate.astype(np.float64)).T + np.abs(inp.bias)
        assert (np.abs(got - ref) <= (d + 8) * 2.0 ** -24 * mag).all()
    B().bfmoe_check_device_error()


CASES = [("sigmoid groups", 64, 16, 3, 70, "f32", dict(score="sigmoid", n_groups=4, top_groups=2, group_score="top2",
                                                       renormalize=True, scale=2.5)),
         ("plain softmax", 64, 8, 2, 37, "f32", dict(score="softmax", renormalize=False)),
         ("softmax bf16", 128, 32, 4, 129, "bf16", dict(score="softmax", renormalize=True, scale=1.5))]


def okw(sc):
    return dict(score=sc.score, groups=sc.n_groups, top_groups=sc.top_groups, group_score=sc.group_score,
                renorm=sc.renormalize, scale=sc.scale)


@pytest.mark.parametrize("name,d,N,k,T,dtype,how", CASES, ids=[c[0] for c in CASES])
def test_layer_object(name, d, N, k, T, dtype, how):
    inp, layer, x, wg, bias = setup(d, N, k, T, dtype, 3)
    sc = B().Scoring(**how)
    bb = np.random.default_rng(0).normal(size=N).astype(np.float32) * 0.1
    xdt = torch.bfloat16 if dtype == "bf16" else torch.float32
    moe = B().ButterflyMoE(layer, wg, bias, k, T + 3, xdt, scoring=sc, balance_bias=torch.from_numpy(bb).cuda())
    y = moe(x).clone()
    logits = moe.logits[:T].double().cpu().numpy()
    idx, gates = S.route(logits, k, bias=bb, **okw(sc))
    assert np.array_equal(moe.idx[:T].cpu().numpy(), idx)
    ref = O.forward_tokens(inp.x_f64(), inp.w_base, inp.alpha, inp.theta, inp.phi, idx, gates)
    tol = 1e-2 if dtype == "bf16" else 1e-5
    assert O.rel_l2_per_token(y.double().cpu().numpy(), ref).max() <= tol
    yd = moe.decode(x).double().cpu().numpy()
    assert O.rel_l2_per_token(yd, ref).max() <= (2.5e-3 if dtype == "bf16" else 1e-5)
    with pytest.raises(ValueError):
        moe.forward_host(x.cpu(), x.cpu())
    with pytest.raises(ValueError):
        B().ButterflyMoE(layer, wg, bias, k, T, xdt, balance_bias=wg[0])
    B().bfmoe_check_device_error()


@pytest.mark.parametrize("name,d,N,k,T,dtype,how", CASES, ids=[c[0] for c in CASES])
def test_training_step(name, d, N, k, T, dtype, how):
    """One step, every gradient, then the clip; the router's remaining products by torch."""
    m = B()
    inp, layer, x, wg, bias = setup(d, N, k, T, dtype, 4)
    sc = m.Scoring(**how)
    rng = np.random.default_rng(1)
    gy = rng.normal(size=(T, d)).astype(np.float32)
    dl = torch.tensor([0.2, 0.05], device="cuda")
    logits = m.bfmoe_router_logits(x, wg, bias)
    routing = m.bfmoe_route(logits, k, sc)
    loss, load = m.bfmoe_balance_loss(logits, routing[0], sc.score)
    g = m.bfmoe_expert_backward(layer, x, k, routing, torch.from_numpy(gy).cuda())
    dlogits = m.bfmoe_route_backward(logits, routing[0], sc, dgates=g["dgates"], load=load, dloss=dl)
    dwg = dlogits.t() @ x.float()
    db = dlogits.sum(0)
    dx = g["dx"] + dlogits @ wg
    m.bfmoe_check_device_error()
    # the oracle on the routing of the same logits
    l64 = logits.double().cpu().numpy()
    idx, gates = S.route(l64, k, **okw(sc))
    assert np.array_equal(routing[0].cpu().numpy(), idx)
    xs = inp.x_f64()
    gy64 = gy.astype(np.float64)
    ref_dg = np.zeros((T, k))
    for j in range(k):
        one = O.forward_tokens(xs, inp.w_base, inp.alpha, inp.theta, inp.phi, idx[:, j:j + 1], np.ones((T, 1)))
        ref_dg[:, j] = (one * gy64).sum(1)
    tol = 2e-4  # of the largest value, as for bfmoe_backward
    assert np.abs(g["dgates"].cpu().numpy() - ref_dg).max() <= tol * np.abs(ref_dg).max()
    (bal, z), lo, rows = S.balance_loss(l64, idx, sc.score)
    assert np.allclose(loss.cpu().numpy(), (bal, z), rtol=1e-5)
    ref_dl, _ = S.route_backward(l64, idx, score=sc.score, renorm=sc.renormalize, scale=sc.scale, dgates=ref_dg,
                                 load=lo, rows=rows, dloss=(float(dl[0]), float(dl[1])))
    assert np.abs(dlogits.cpu().numpy() - ref_dl).max() <= tol * np.abs(ref_dl).max()
    # dx of the experts by differences of the oracle's forward, gates held
    u = rng.normal(size=xs.shape)
    h = 1e-6
    up = O.forward_tokens(xs + h * u, inp.w_base, inp.alpha, inp.theta, inp.phi, idx, gates)
    dn = O.forward_tokens(xs - h * u, inp.w_base, inp.alpha, inp.theta, inp.phi, idx, gates)
    num = ((up - dn) * gy64).sum() / (2 * h)
    got = float((g["dx"].double().cpu().numpy() * u).sum())
    assert abs(num - got) <= 1e-4 * np.abs(g["dx"].double().cpu().numpy() * u).sum()
    # clip the layer's list
    grads = [g["dtheta"], g["dphi"], g["dw_base"], g["dalpha"], dwg.contiguous(), db, dx.contiguous()]
    ref = S.grad_norm([t.double().cpu().numpy() for t in grads])
    norm = m.bfmoe_grad_clip(grads, 1.0)
    assert abs(float(norm) - ref) <= 1e-6 * ref
    after = S.grad_norm([t.double().cpu().numpy() for t in grads])
    assert abs(after - min(1.0, ref)) <= 1e-6


def test_readme_example_clips_every_step():
    """The README's Python example, its training part three times over (what is marked as made once: once)."""
    m = B()
    with open(os.path.join(os.path.dirname(__file__), "..", "README.md")) as f:
        text = f.read()
    code = text[text.index("```python") + len("```python"):]
    first, step = code[:code.index("```")].split("# the same in a training step")
    inp, _, x, wg, bias = setup(64, 16, 2, 40, "bf16", 5)
    host = x.cpu().pin_memory()
    env = dict(torch=torch, w_base_int8=inp.w_base, alpha=inp.alpha, theta=inp.theta, phi=inp.phi, w_gate=wg, bias=bias,
               k=2, max_tokens=64, x=x, x_small=x[:3].contiguous(), x_pinned=host, y_pinned=torch.empty_like(host).pin_memory(),
               bb=torch.randn(16, device="cuda") * 0.1, gy=torch.randn(40, 64, device="cuda"),
               dloss=torch.tensor([0.01, 0.001], device="cuda"))
    exec(first, env)
    step = step[step.index("\n"):]
    for i in range(3):
        env["gy"] = torch.randn(40, 64, device="cuda") * (i + 1)
        exec("\n".join(l for l in step.split("\n") if i == 0 or "made once" not in l), env)
        g = env["grads"]
        after = S.grad_norm([g[n].double().cpu().numpy() for n in ("dtheta", "dphi", "dw_base")])
        assert float(env["norm"]) > 1 and abs(after - 1) <= 1e-6, (i, float(env["norm"]), after)
    m.bfmoe_check_device_error()


def test_expert_backward_is_backward_without_the_router():
    """With plain softmax gates, bfmoe_expert_backward + bfmoe_route_backward + products equal bfmoe_backward."""
    m = B()
    d, N, k, T = 64, 8, 2, 90
    inp, layer, x, wg, bias = setup(d, N, k, T, "f32", 6)
    gy = torch.randn(T, d, device="cuda")
    ws = m.workspace(d, N, T, k, m.BFMOE_F32)
    routing = m.bfmoe_router_topk(x, wg, bias, k, ws)
    a = m.bfmoe_backward(layer, x, k, wg, routing, gy)
    b = m.bfmoe_expert_backward(layer, x, k, routing, gy)
    logits = m.bfmoe_router_logits(x, wg, bias)
    dlog = m.bfmoe_route_backward(logits, routing[0], m.Scoring(), dgates=b["dgates"])
    for key in ("dw_base", "dalpha"):
        assert torch.equal(a[key], b[key])
    pairs = [(a[q], b[q]) for q in ("dtheta", "dphi")]
    pairs += [(a["dx"], b["dx"] + dlog @ wg), (a["dw_gate"], dlog.t() @ x), (a["dbias"], dlog.sum(0))]
    for p, q in pairs:
        assert float((p - q).abs().max()) <= 2e-5 * float(p.abs().max())
