"""Routing, its gradient and its losses where a warp takes many rows one after the other (rows loaded ahead, two
buffers used in turn, chosen terms cleared between rows, rows left for the end), against plain float64 forms of all
rows.  A warp takes a second row above about 3500 rows; the sizes give it five and more, the last step ragged.

Tolerances as in test_gpu_route.py: (64 + 4 max|l|) half steps of float32 of the magnitudes that a value is summed
from, and half a step of bfloat16 for a bfloat16 gradient.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HALF = 2.0 ** -24
TINY = 1e-37
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import ternary_butterfly_experts_b200.build as b
    b.build()


def B():
    import ternary_butterfly_experts_b200 as m
    return m


def steps(l):
    return (64 + 4 * float(l[l.abs() < 1e30].abs().max())) * HALF


def make(T, N, dtype, seed, off=0, special=True):
    """Logits on the GPU (rows ``off`` elements into rows of N + 2 off), rows of equal, masked and few logits among
    them, and their float64 values (NaN as -inf)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    l = torch.randn(T, N, generator=g, device="cuda") * 1.5 + torch.randn(N, generator=g, device="cuda")
    if special:
        l[3::7] = 0.25                      # equal logits: more candidates than lanes
        l[5::1000] = -INF
        l[6::1000, : N - 2] = -INF          # fewer than k left
        l[8::1000, ::3] = float("nan")
    big = torch.zeros(T, N + 2 * off, device="cuda", dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
    x = big[:, off:off + N]
    x.copy_(l)
    v = x.double()
    return x, torch.where(v > -INF, v, -INF)


def scores(l, score):
    live = l > -INF
    if score == "sigmoid":
        return torch.where(live, torch.sigmoid(l), 0.0)
    top = l.amax(1, keepdim=True)
    e = torch.where(live, torch.exp(l - top), 0.0)
    return e / e.sum(1, keepdim=True).clamp(min=1e-300)


def plain_route(l, k, score, bias=None, groups=1, top_groups=1, renorm=True, scale=1.0):
    T, N = l.shape
    live = l > -INF
    s = scores(l, score)
    value = torch.where(live, l if bias is None else s + bias.double(), -1e300)
    if top_groups < groups:
        best = torch.where(live, s if bias is None else s + bias.double(), -INF).view(T, groups, -1).topk(2, -1)[0]
        worth = torch.where(best[..., 1] > -INF, best.sum(-1), best[..., 0])
        kept = worth.sort(dim=1, descending=True, stable=True)[1][:, :top_groups]
        keep = torch.zeros_like(worth, dtype=torch.bool).scatter_(1, kept, True)
        value = torch.where(keep.repeat_interleave(N // groups, 1), value, -INF)
    e = value.sort(dim=1, descending=True, stable=True)[1][:, :k]
    g = s.gather(1, e)
    if renorm:
        g = g / g.sum(1, keepdim=True).clamp(min=1e-300)
    return e, g * scale


def check_buckets(idx, out, N):
    flat = idx.reshape(-1)
    counts = torch.bincount(flat, minlength=N)
    assert torch.equal(out[2].long(), counts)
    assert torch.equal(out[3].long(), torch.cat([counts.new_zeros(1), counts.cumsum(0)]))
    assert torch.equal(out[4].long(), flat.sort(stable=True)[1])


KINDS = [dict(score="softmax"), dict(score="softmax", renorm=False), dict(score="sigmoid", bias=True, scale=2.5),
         dict(score="softmax", bias=True), dict(score="sigmoid", bias=True, groups=4, top_groups=2)]


@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,k", [(20011, 512, 4), (20011, 1000, 3), (20011, 1024, 8), (40003, 264, 8),
                                   (20011, 256, 8), (40003, 64, 2)])
def test_route(T, N, k, dtype, off):
    x, l = make(T, N, dtype, T + N, off)
    for kind in KINDS:
        kw = dict(kind)
        bias = torch.randn(N, device="cuda", generator=torch.Generator(device="cuda").manual_seed(N)) * 0.1
        bias = bias if kw.pop("bias", False) else None
        sc = B().Scoring(kw["score"], n_groups=kw.get("groups", 1), top_groups=kw.get("top_groups", 1),
                         group_score="top2", renormalize=kw.get("renorm", True), scale=kw.get("scale", 1.0))
        out = B().bfmoe_route(x, k, sc, balance_bias=bias)
        B().bfmoe_check_device_error()
        e, g = plain_route(l, k, bias=bias, **kw)
        bad = (out[0].long() != e).any(1).nonzero()[:, 0]
        assert bad.numel() == 0, (kind, bad[:5], out[0][bad[:3]], e[bad[:3]])
        assert ((out[1].double() - g).abs() <= steps(l) * g.abs() + TINY).all()
        check_buckets(e, out, N)


def plain_load(l, e, score):
    some = (l > -INF).any(1)
    load = torch.bincount(e[some].reshape(-1), minlength=l.shape[1])
    return some, load


def shares(l, score):
    s = scores(l, score)
    return s / s.sum(1, keepdim=True).clamp(min=1e-300)


def plain_backward(l, e, score, renorm, scale, dg, load, rows, dl):
    """(gradient, sum of the magnitudes of its terms) of every row."""
    T, N = l.shape
    k = e.shape[1]
    live = l > -INF
    s = scores(l, score)
    g, b = torch.zeros_like(l), torch.zeros_like(l)
    if dg is not None:
        d = dg.double() * scale * torch.gather(live, 1, e)
        if score == "softmax" and not renorm:
            t = s.gather(1, e) * d
            g -= s * t.sum(1, keepdim=True)
            b += s * t.abs().sum(1, keepdim=True)
            g.scatter_add_(1, e, t)
            b.scatter_add_(1, e, t.abs())
        else:
            if renorm:
                r = s.gather(1, e)
                r = r / r.sum(1, keepdim=True).clamp(min=1e-300)
                t, m = r * (d - (r * d).sum(1, keepdim=True)), r * (d.abs() + (r * d).abs().sum(1, keepdim=True))
            else:
                t = s.gather(1, e) * d
                m = t.abs()
            if score == "sigmoid":
                f = torch.where(live, torch.sigmoid(-l), 0.0).gather(1, e)
                t, m = t * f, m * f
            g.scatter_add_(1, e, t)
            b.scatter_add_(1, e, m)
    if load is not None:
        f = load.double() / (k * rows)
        p = shares(l, score)
        fp = (p * f).sum(1, keepdim=True)
        w = torch.where(live, torch.sigmoid(-l), 0.0) if score == "sigmoid" else 1.0
        g += dl[0] * N / rows * p * (f - fp) * w
        b += abs(dl[0]) * N / rows * p * (f + fp) * w
        if dl[1]:
            lse = torch.logsumexp(l, 1, keepdim=True)
            q = torch.where(live, scores(l, "softmax") * lse, 0.0) * (2 * dl[1] / rows)
            g += q
            b += q.abs()
    return g, b


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,k,off", [(40003, 64, 2, 0), (40003, 128, 4, 0), (40003, 120, 3, 1), (40003, 256, 8, 0),
                                       (40003, 250, 8, 0), (40003, 256, 2, 3), (20011, 500, 4, 0), (20011, 1024, 4, 0),
                                       (20011, 1000, 8, 1)])
def test_backward(T, N, k, off, dtype, in_place):
    for score, renorm, gates, losses in (("softmax", False, True, (0.3, 0.7)), ("sigmoid", True, True, (0.3, 0.7)),
                                         ("softmax", False, True, None), ("softmax", True, True, None),
                                         ("sigmoid", False, True, (0.5, 0.0)), ("softmax", True, False, (0.2, 0.1))):
        x, l = make(T, N, dtype, T + N + k, off)
        e, _ = plain_route(l, k, score)
        dg = torch.randn(T, k, device="cuda") if gates else None
        kw, load, rows = {}, None, 0
        if losses:
            some, load = plain_load(l, e, score)
            rows = int(some.sum())
            kw = dict(load=torch.cat([load, load.new_tensor([rows])]).int(),
                      dloss=torch.tensor(losses, dtype=torch.float32, device="cuda"))
            losses = [float(v) for v in kw["dloss"]]
        out = None
        if in_place:
            out = x
        got = B().bfmoe_route_backward(x, e.int(), B().Scoring(score, renormalize=renorm, scale=1.5), dgates=dg,
                                       dlogits=out, **kw)
        B().bfmoe_check_device_error()
        want, bound = plain_backward(l, e, score, renorm, 1.5, dg, load, rows, losses)
        err = (got.double() - want).abs()
        lim = steps(l) * bound + TINY
        if dtype == "bf16":
            lim = lim + 2.0 ** -8 * (want.abs() + lim)
        assert (err <= lim).all(), (score, renorm, gates, losses, float((err - lim).max()))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,k,off", [(40003, 64, 2, 0), (40003, 128, 4, 0), (40003, 256, 8, 0), (40003, 250, 8, 0),
                                       (40003, 512, 2, 1), (40003, 1024, 4, 0)])
def test_losses(T, N, k, off, dtype):
    x, l = make(T, N, dtype, T + N + k + 1, off)
    for score in ("softmax", "sigmoid"):
        e, _ = plain_route(l, k, score)
        loss, load = B().bfmoe_balance_loss(x, e.int(), score)
        B().bfmoe_check_device_error()
        some, ref = plain_load(l, e, score)
        rows = int(some.sum())
        assert torch.equal(load[:N].long(), ref) and int(load[N]) == rows
        bal = float(N * (ref.double() / (k * rows) * shares(l, score)[some].sum(0) / rows).sum())
        z = float(torch.logsumexp(l[some], 1).square().mean())
        got = loss.double().tolist()
        assert abs(got[0] - bal) <= steps(l) * bal
        assert abs(got[1] - z) <= 2 * steps(l) * (z + z ** 0.5)
        for _ in range(2):  # the same sums in the same order
            again = B().bfmoe_balance_loss(x, e.int(), score)
            assert torch.equal(again[0], loss) and torch.equal(again[1], load)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,k,off", [(40003, 64, 2, 0), (40003, 128, 4, 0), (40003, 256, 2, 0), (20011, 250, 4, 0),
                                       (20011, 512, 4, 0), (20011, 1024, 4, 0), (20011, 1000, 3, 1)])
def test_backward_goes_on_behind_rows_that_are_not_finite(T, N, k, off, dtype, in_place):
    """Rows with a +inf logit under a z loss, and with a NaN gate gradient, here and there: every other row is as
    ever, also those that their warp had on the way."""
    x, l = make(T, N, dtype, T + N, off, special=False)
    inf_rows = torch.arange(17, T, 1501, device="cuda")
    nan_rows = torch.arange(801, T, 1501, device="cuda")
    e, _ = plain_route(l, k, "softmax")
    x[inf_rows, 5] = INF
    dg = torch.randn(T, k, device="cuda")
    dg[nan_rows, 0] = float("nan")
    load, losses = torch.bincount(e.reshape(-1), minlength=N), (0.3, 0.7)
    dl = torch.tensor(losses, dtype=torch.float32, device="cuda")
    losses = [float(v) for v in dl]
    got = B().bfmoe_route_backward(x, e.int(), B().Scoring("softmax", renormalize=False), dgates=dg, dloss=dl,
                                   load=torch.cat([load, load.new_tensor([T])]).int(), dlogits=x if in_place else None)
    B().bfmoe_check_device_error()
    got = got.double()
    assert torch.isinf(got[inf_rows, 5]).all() and torch.isnan(got[nan_rows]).all()
    rest = torch.ones(N, dtype=torch.bool, device="cuda")
    rest[5] = False
    # nothing reaches the others of a +inf row but their own gate's term, which is 0 times it
    assert (got[inf_rows][:, rest] == 0).all()
    ok = torch.ones(T, dtype=torch.bool, device="cuda")
    ok[inf_rows] = ok[nan_rows] = False
    want, bound = plain_backward(l, e, "softmax", False, 1.0, dg.nan_to_num(), load, T, losses)
    lim = steps(l) * bound + TINY
    if dtype == "bf16":
        lim = lim + 2.0 ** -8 * (want.abs() + lim)
    assert ((got - want).abs() <= lim)[ok].all()
