"""Routing from logits, its gradient and its losses through the C ABI against
the float64 oracle (oracle/scored_oracle.py, pinned by test_scored_oracle.py).

Experts and buckets must equal the oracle's.  Gates and gradients are float32
arithmetic: exp(x) carries |x| half steps of its argument (|x| <= twice the
largest finite logit) and the sums of up to N positive terms a few dozen more,
so a value is off by at most (64 + 4 max|l|) half steps of float32 of the
magnitudes it is summed from; a bfloat16 gradient adds half a step of its own.
"""
import numpy as np
import pytest

from oracle import bfmoe_oracle as O
from oracle import scored_oracle as S

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HALF = float(torch.finfo(torch.float32).eps) / 2
TINY = 1e-37  # below the smallest normal float32: what flushes to zero


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import ternary_butterfly_experts_b200.build as b
    b.build()


def B():
    import ternary_butterfly_experts_b200 as m
    return m


def half_steps(l):
    fin = np.abs(l[np.isfinite(l)])
    # logits that a mask sets to the lowest value meet only exp(0) and exp(-huge) = 0
    fin = fin[fin < 1e30]
    return (64 + 4 * (fin.max() if fin.size else 0.0)) * HALF


def make_logits(T, N, dtype, seed, std=1.5):
    rng = np.random.default_rng(seed)
    l = (rng.normal(size=(T, N)) + 0.7 * rng.normal(size=N)) * std
    t = torch.from_numpy(l).to(torch.float32).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    return t, t.double().numpy()


def scoring(score="softmax", groups=1, top_groups=1, group_score="max", renorm=True, scale=1.0):
    return B().Scoring(score=score, n_groups=groups, top_groups=top_groups, group_score=group_score,
                       renormalize=renorm, scale=scale)


def check_route(t, l, k, bias=None, buckets=True, dev_logits=None, **kw):
    """Route t (a CPU tensor, l its float64 values) and compare with the oracle."""
    x = t.cuda() if dev_logits is None else dev_logits
    b = None if bias is None else torch.from_numpy(bias).cuda()
    out = B().bfmoe_route(x, k, scoring(**kw), balance_bias=b, buckets=buckets)
    B().bfmoe_check_device_error()
    idx, gates = out[0].cpu().numpy(), out[1].cpu().numpy().astype(np.float64)
    ref, g = S.route(l, k, bias=bias, **kw)
    bad = np.nonzero((idx != ref).any(1))[0]
    assert bad.size == 0, (bad[:5], idx[bad[:3]], ref[bad[:3]])
    assert np.isfinite(gates).all()
    assert (np.abs(gates - g) <= half_steps(l) * np.abs(g) + TINY * kw.get("scale", 1.0)).all(), np.abs(gates - g).max()
    if buckets:
        counts, offsets, rows = O.buckets(ref, l.shape[1])
        for got, want in zip(out[2:], (counts, offsets, rows)):
            assert np.array_equal(got.cpu().numpy(), want)
    else:
        assert out[2] is None and out[3] is None and out[4] is None
    return out


SHAPES = [(1, 1, 1), (5, 2, 2), (7, 8, 8), (37, 8, 2), (33, 31, 3), (64, 32, 8), (129, 33, 1), (300, 64, 2),
          (70, 100, 6), (129, 128, 4), (41, 250, 8), (257, 256, 8), (65, 257, 5), (40, 512, 7), (31, 1000, 4),
          (130, 1024, 4), (9, 1025, 8), (17, 2500, 3), (12, 4096, 8)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,k", SHAPES)
def test_route_sizes(T, N, k, dtype):
    t, l = make_logits(T, N, dtype, T + N + k)
    bias = np.random.default_rng(N).normal(size=N).astype(np.float32) * 0.1
    check_route(t, l, k)
    check_route(t, l, k, score="softmax", bias=bias, renorm=False, scale=1.7)
    check_route(t, l, k, score="sigmoid", renorm=False)
    check_route(t, l, k, score="sigmoid", bias=bias, scale=2.5, buckets=False)


GROUPS = [(40, 256, 8, 8, 4), (33, 64, 2, 4, 2), (21, 24, 5, 3, 2), (19, 60, 4, 5, 1), (50, 250, 8, 10, 3),
          (9, 64, 4, 64, 9), (7, 1024, 8, 16, 2), (11, 4096, 8, 32, 5), (13, 96, 3, 48, 2), (5, 16, 8, 2, 1),
          (6, 512, 8, 2, 1), (30, 8, 1, 8, 1), (40, 256, 8, 16, 4), (20, 64, 8, 16, 5), (20, 1024, 8, 64, 3)]


@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,N,k,G,top", GROUPS)
def test_route_groups(T, N, k, G, top, score, group_score):
    t, l = make_logits(T, N, "f32", T + N + G)
    bias = np.random.default_rng(G).normal(size=N).astype(np.float32) * 0.2
    kw = dict(score=score, groups=G, top_groups=top, group_score=group_score)
    check_route(t, l, k, bias=bias, **kw)
    check_route(t, l, k, renorm=False, **kw)
    t, l = make_logits(T, N, "bf16", T + N + G + 1)
    check_route(t, l, k, bias=bias, **kw)
    check_route(t, l, k, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("N", [4, 40, 256, 1024, 1500])
def test_route_masked_rows(N, score):
    """Rows with no expert left, with fewer than k, with NaN, +inf and the type's lowest value."""
    k = 4
    for dtype in ("f32", "bf16"):
        t, _ = make_logits(12, N, dtype, N)
        low = torch.finfo(t.dtype).min
        t[0] = float("-inf")
        t[1] = float("nan")
        t[2] = low
        t[3] = float("-inf")
        t[3, N // 2] = -3.0
        t[4, ::2] = float("-inf")
        t[5, 1::2] = float("nan")
        t[6, N - 1] = float("inf")
        t[7, : N // 2] = float("inf")
        t[8] = low
        t[8, N - 2] = 0.25
        t[9] = -200.0
        t[9, 1] = -201.0
        t[10] = 90.0
        t[11, : N - 1] = float("-inf")
        l = t.double().numpy()
        bias = np.random.default_rng(3).normal(size=N).astype(np.float32)
        off = bias.copy()
        off[::3] = -np.inf
        off[1] = np.nan
        for renorm in (True, False):
            check_route(t, l, k, score=score, renorm=renorm)
            check_route(t, l, k, score=score, renorm=renorm, bias=bias)
            check_route(t, l, k, score=score, renorm=renorm, bias=off)
            for gs in ("max", "top2"):
                check_route(t, l, 2, score=score, renorm=renorm, bias=off, groups=2, top_groups=1, group_score=gs)
                check_route(t, l, 2, score=score, renorm=renorm, groups=2, top_groups=1, group_score=gs)


@pytest.mark.parametrize("N,G", [(8, 2), (64, 4), (256, 8), (1024, 16), (2048, 8)])
def test_route_ties(N, G):
    """Equal logits everywhere, few distinct values, and equal biases: the lower index wins."""
    bias = np.zeros(N, np.float32)
    for dtype in ("f32", "bf16"):
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        zero = torch.zeros(9, N, dtype=dt)
        few = torch.randint(-2, 3, (40, N), generator=torch.Generator().manual_seed(N)).to(dt)
        signed = torch.where(few > 0, torch.zeros_like(few), -torch.zeros_like(few))  # 0 and -0 are equal
        for t in (zero, few, signed):
            l = t.double().numpy()
            for score in ("softmax", "sigmoid"):
                check_route(t, l, 8, score=score)
                check_route(t, l, 8, score=score, bias=bias)
                check_route(t, l, 4, score=score, bias=bias, groups=G, top_groups=G // 2, group_score="top2")
                check_route(t, l, 4, score=score, groups=G, top_groups=G // 2, group_score="max")


@pytest.mark.parametrize("N", [64, 256, 1024, 1300])
def test_route_near_ties(N):
    """Values that float32 cannot rank, 1e-9 apart in 64 bits: the choice is the 64-bit one."""
    rng = np.random.default_rng(N)
    T, k = 24, 6
    l = rng.normal(size=(T, N)).astype(np.float32)
    # a bias that makes the sigmoid values of row 0 nearly equal to 0.9 for half the experts
    s = 1 / (1 + np.exp(-l[0].astype(np.float64)))
    bias = (0.9 - s).astype(np.float32)
    bias[N // 2:] -= 5
    l[1:] = l[0]
    for t in range(1, T):  # neighbouring float32 logits: steps of one unit in the last place
        l[t] = np.nextafter(l[0], np.float32(10 if t % 2 else -10))
        l[t, rng.integers(0, N, 5)] += np.float32(3e-7)
    check_route(torch.from_numpy(l), l.astype(np.float64), k, score="sigmoid", bias=bias)
    check_route(torch.from_numpy(l), l.astype(np.float64), k, score="softmax", bias=bias * 1e-3)
    check_route(torch.from_numpy(l), l.astype(np.float64), 2, score="sigmoid", bias=bias, groups=4, top_groups=2,
                group_score="top2")
    # logits one unit in the last place apart: no bias, exact order
    base = np.float32(1.7)
    up = np.full((3, N), base, np.float32)
    up[0, N - 3] = np.nextafter(base, np.float32(2))
    up[1, 5:] = np.nextafter(base, np.float32(0))
    up[2] = (base + np.arange(N) * np.float32(1.2e-7)).astype(np.float32)
    for kw in (dict(), dict(score="sigmoid", renorm=False)):
        check_route(torch.from_numpy(up), up.astype(np.float64), 8, **kw)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("N,G", [(64, 32), (64, 4), (120, 5), (256, 8), (256, 64), (1000, 10), (1024, 16), (2048, 16)])
def test_route_near_groups_of_terms_that_cancel(N, G, score):
    """Two experts a group, with biases of +1000 and -1000: float32 rounds each value by 3e-5, 64 bits rank sums that
    are nearer than that."""
    rng = np.random.default_rng(N + G)
    T, per = 64, N // G
    l = np.full((T, N), -np.inf, np.float32)
    bias = np.zeros(N, np.float32)
    spread = 3e-4 if score == "sigmoid" else 2e-4 * G   # of the logits: 7e-5 and more of the scores
    for g in range(G):
        a, b = g * per, g * per + per // 2 if per > 2 else g * per + 1
        l[:, a] = rng.normal(size=T) * spread
        l[:, b] = rng.normal(size=T) * spread
        bias[a], bias[b] = 1000, -1000
    check_route(torch.from_numpy(l), l.astype(np.float64), 2, score=score, bias=bias, groups=G, top_groups=G // 2,
                group_score="top2")


@pytest.mark.parametrize("N", [16, 64, 100, 256, 1024, 2048])
def test_route_groups_of_the_lowest_value(N):
    """Two biases of the type's lowest value leave float32 when they are added up; such a group still comes before
    one that has no expert left."""
    per = N // 4
    t, _ = make_logits(5, N, "f32", N)
    t[:, : 2 * per] = float("-inf")
    t[:, 3 * per + 3:] = float("-inf")
    bias = np.zeros(N, np.float32)
    bias[2 * per:3 * per] = np.finfo(np.float32).min
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            check_route(t, t.double().numpy(), 4, score=score, renorm=renorm, bias=bias, groups=4, top_groups=2,
                        group_score="top2")


@pytest.mark.parametrize("shift", [-300.0, 25.0, 400.0, 5000.0])
def test_route_shifted_logits(shift):
    """A shift of every logit changes no softmax; near values are ranked as in 64 bits all the same."""
    for N in (64, 256, 1024):
        rng = np.random.default_rng(N)
        l = (rng.normal(size=(60, N)) + shift).astype(np.float32)
        p = np.exp(l[0].astype(np.float64) - l[0].max())
        bias = (0.3 - p / p.sum()).astype(np.float32)   # row 0: every value next to 0.3
        l[1:] = l[0]
        l[np.arange(1, 60), rng.integers(0, N, 59)] += np.float32(1e-3)
        check_route(torch.from_numpy(l), l.astype(np.float64), 6, bias=bias, renorm=False)
        check_route(torch.from_numpy(l), l.astype(np.float64), 6, score="sigmoid", bias=bias)
        check_backward(torch.from_numpy(l[:9]), l[:9].astype(np.float64), 3, "softmax", False, 1.0)
        check_backward(torch.from_numpy(l[:9]), l[:9].astype(np.float64), 3, "sigmoid", True, 1.0)


def test_route_strided_and_unaligned_rows():
    for dtype in (torch.float32, torch.bfloat16):
        for N, ld, off in ((256, 300, 1), (64, 67, 3), (250, 256, 2), (1024, 1029, 5), (1500, 1501, 1)):
            big = torch.randn(50, ld + off, generator=torch.Generator().manual_seed(ld)).to(dtype)
            t = big[:, off:off + N]
            dev = big.cuda()[:, off:off + N]
            assert not dev.is_contiguous()
            check_route(t, t.double().numpy(), 5, dev_logits=dev)


def test_route_offsets_past_32_bits():
    """70000 rows 40000 elements apart: the last ones start 2.8e9 elements in."""
    T, N, ld = 70000, 16, 40000
    big = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda")
    v = big.view(T, ld)[:, :N]
    t, l = make_logits(T, N, "bf16", 1)
    v.copy_(t.cuda())
    sc = scoring("sigmoid")
    idx, gates = B().bfmoe_route(v, 3, sc, buckets=False)[:2]
    tail = slice(T - 40, T)
    ref, g = S.route(l[tail], 3, score="sigmoid")
    assert np.array_equal(idx[tail].cpu().numpy(), ref)
    d = torch.zeros_like(big).view(T, ld)[:, :N]
    dg = torch.randn(T, 3, device="cuda")
    B().bfmoe_route_backward(v, idx, sc, dgates=dg, dlogits=d)
    want, bound = S.route_backward(l[tail], ref, score="sigmoid", dgates=dg[tail].cpu().numpy())
    assert (np.abs(d[tail].double().cpu().numpy() - want) <= half_steps(l) * bound + 2.0 ** -8 * np.abs(want) + TINY).all()
    B().bfmoe_check_device_error()


def test_route_empty_batch():
    x = torch.empty(0, 16, device="cuda")
    idx, gates, counts, offsets, rows = B().bfmoe_route(x, 2, scoring())
    assert idx.shape == (0, 2) and rows.numel() == 0
    assert int(counts.sum()) == 0 and int(offsets.abs().sum()) == 0
    loss, load = B().bfmoe_balance_loss(x, idx)
    assert loss.tolist() == [0.0, 0.0] and int(load.sum()) == 0
    assert B().bfmoe_route_backward(x, idx, scoring(), dgates=gates).shape == (0, 16)


def test_route_is_deterministic_and_leaves_the_rest_alone():
    t, l = make_logits(700, 256, "f32", 9)
    x = t.cuda()
    sc = scoring("sigmoid", groups=8, top_groups=4, group_score="top2", scale=2.5)
    bias = torch.randn(256, device="cuda") * 0.1
    a = B().bfmoe_route(x, 8, sc, balance_bias=bias)
    # outputs with room behind them: what is behind stays as it was
    idx = torch.full((705, 8), -7, dtype=torch.int32, device="cuda")
    gates = torch.full((705, 8), -7.0, device="cuda")
    rows = torch.full((705 * 8,), -7, dtype=torch.int32, device="cuda")
    out = (idx[:700], gates[:700], torch.empty_like(a[2]), torch.empty_like(a[3]), rows[:5600])
    b = B().bfmoe_route(x, 8, sc, balance_bias=bias, out=out)
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    assert (idx[700:] == -7).all() and (gates[700:] == -7).all() and (rows[5600:] == -7).all()
    assert torch.equal(x, t.cuda())


def test_route_graph_and_streams():
    """Captured, replayed on new values, on a stream of its own, next to an eager call on another stream."""
    T, N, k = 513, 256, 8
    sc = scoring("sigmoid", groups=8, top_groups=4, group_score="top2")
    t1, l1 = make_logits(T, N, "f32", 1)
    t2, l2 = make_logits(T, N, "f32", 2)
    x = t1.cuda()
    n = B().bfmoe_route_workspace_size(N, T, k)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(n, dtype=torch.uint8, device="cuda")
    dg = torch.randn(T, k, device="cuda")
    dl = torch.tensor([0.01, 0.001], device="cuda")

    def step(ws):
        out = B().bfmoe_route(x, k, sc, ws=ws)
        loss, load = B().bfmoe_balance_loss(x, out[0], "sigmoid", ws=ws)
        return (*out, loss, load, B().bfmoe_route_backward(x, out[0], sc, dgates=dg, load=load, dloss=dl))

    step(ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = step(ws)
    x.copy_(t2.cuda())
    g.replay()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.current_stream())
        eager = step(ws2)
    torch.cuda.synchronize()
    for a, b in zip(got, eager):
        assert torch.equal(a, b)
    ref, _ = S.route(l2[:64], k, score="sigmoid", groups=8, top_groups=4, group_score="top2")
    assert np.array_equal(got[0][:64].cpu().numpy(), ref)
    B().bfmoe_check_device_error()


# -------------------------------------------------------------------------------------------------------------------
# gradient
# -------------------------------------------------------------------------------------------------------------------
def check_backward(t, l, k, score, renorm, scale, gates=True, aux=True, idx=None, z=0.7, in_place=False):
    T, N = l.shape
    if idx is None:
        idx, _ = S.route(l, k, score=score)
    rng = np.random.default_rng(T + N)
    x = t.cuda()
    di = torch.from_numpy(np.ascontiguousarray(idx, np.int32)).cuda()
    dg = rng.normal(size=(T, k)).astype(np.float32) if gates else None
    kw, okw = {}, {}
    if aux:
        _, load, rows = S.balance_loss(l, idx, score)
        dl = np.array([0.3, z], np.float32)
        kw = dict(load=torch.from_numpy(np.append(load, rows).astype(np.int32)).cuda(), dloss=torch.from_numpy(dl).cuda())
        okw = dict(load=load, rows=rows, dloss=tuple(float(v) for v in dl))
    out = x if in_place else None
    got = B().bfmoe_route_backward(x, di, scoring(score, renorm=renorm, scale=scale),
                                   dgates=None if dg is None else torch.from_numpy(dg).cuda(), dlogits=out, **kw)
    B().bfmoe_check_device_error()
    assert got.dtype == t.dtype and (not in_place or got.data_ptr() == x.data_ptr())
    want, bound = S.route_backward(l, idx, score=score, renorm=renorm, scale=scale, dgates=dg, **okw)
    step = float(torch.finfo(t.dtype).eps) / 2 if t.dtype == torch.bfloat16 else 0.0
    err = np.abs(got.double().cpu().numpy() - want)
    lim = half_steps(l) * bound + step * (np.abs(want) + half_steps(l) * bound) + TINY
    assert (err <= lim).all(), (err - lim).max()
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,k", SHAPES)
def test_backward_sizes(T, N, k, dtype):
    t, l = make_logits(T, N, dtype, T + N + 5)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            check_backward(t, l, k, score, renorm, 2.5)
        check_backward(t, l, k, score, True, 1.0, aux=False)
        check_backward(t, l, k, score, False, 1.0, aux=False)
        check_backward(t, l, k, score, True, 1.0, gates=False)
        check_backward(t, l, k, score, False, 1.5, in_place=True)


@pytest.mark.parametrize("N", [6, 64, 256, 1100])
def test_backward_masked_rows(N):
    for dtype in ("f32", "bf16"):
        t, _ = make_logits(8, N, dtype, N + 1)
        t[0] = float("-inf")
        t[1] = float("nan")
        t[2] = torch.finfo(t.dtype).min
        t[3] = float("-inf")
        t[3, N // 2] = -3.0
        t[4, ::2] = float("-inf")
        t[5] = -200.0
        t[6] = 60.0
        l = t.double().numpy()
        for score in ("softmax", "sigmoid"):
            for renorm in (True, False):
                check_backward(t, l, 3, score, renorm, 1.5, z=0.0)
                check_backward(t, l, 3, score, renorm, 1.5, aux=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [6, 64, 250, 256, 1024, 1100])
def test_backward_of_infinite_logits(N, dtype):
    """Logits of +inf share the mass: the others' gradient through the row's sums is 0, masked ones have none at all,
    and only a z loss has an infinite gradient, that of the +inf logits alone."""
    k = 3
    t, _ = make_logits(6, N, dtype, N + 2)
    t[1, N - 1] = float("inf")
    t[2, [0, N // 2, N - 2]] = float("inf")
    t[3, 1::2] = float("-inf")
    t[3, 2] = float("inf")
    t[4] = float("inf")
    t[5, : N - 1] = float("nan")
    t[5, N - 1] = float("inf")
    l = t.double().numpy()
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            check_backward(t, l, k, score, renorm, 1.5, aux=False)
            check_backward(t, l, k, score, renorm, 1.5, z=0.0)
            # with a z loss: infinities where the oracle has them, of its sign, the rest as ever
            idx, _ = S.route(l, k, score=score)
            _, load, rows = S.balance_loss(l, idx, score)
            dg = np.random.default_rng(N).normal(size=(6, k)).astype(np.float32)
            for z in (0.7, -0.7):
                dl = np.array([0.3, z], np.float32)
                got = B().bfmoe_route_backward(
                    t.cuda(), torch.from_numpy(idx.astype(np.int32)).cuda(), scoring(score, renorm=renorm, scale=1.5),
                    dgates=torch.from_numpy(dg).cuda(), dloss=torch.from_numpy(dl).cuda(),
                    load=torch.from_numpy(np.append(load, rows).astype(np.int32)).cuda()).double().cpu().numpy()
                want, bound = S.route_backward(l, idx, score=score, renorm=renorm, scale=1.5, dgates=dg, load=load,
                                               rows=rows, dloss=tuple(float(v) for v in dl))
                inf = np.isinf(want)
                assert (inf == ((l == np.inf) & (np.arange(6) > 0)[:, None])).all()
                assert np.array_equal(got[inf], want[inf])
                lim = half_steps(l) * bound[~inf] + TINY
                if dtype == "bf16":
                    lim = lim + 2.0 ** -8 * (np.abs(want[~inf]) + lim)
                assert (np.abs(got[~inf] - want[~inf]) <= lim).all()


@pytest.mark.parametrize("N", [12, 250, 1024, 1300])
def test_backward_of_gate_gradients_that_are_not_finite(N):
    """A NaN among the gradients of the gates reaches the experts of its row that have a gate; masked experts keep 0,
    chosen ones among them, and so do the other rows."""
    T, k = 5, 4
    t, _ = make_logits(T, N, "f32", N + 4)
    t[:, : N - 3] = float("-inf")
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            sc = scoring(score, renorm=renorm)
            idx, gates = B().bfmoe_route(t.cuda(), k, sc, buckets=False)[:2]
            for bad in (float("nan"), float("inf")):
                dg = torch.randn(T, k, device="cuda")
                dg[2, 0] = bad
                got = B().bfmoe_route_backward(t.cuda(), idx, sc, dgates=dg).cpu()
                assert (got[:, : N - 3] == 0).all(), (score, renorm, bad)
                assert torch.isfinite(got[[0, 1, 3, 4]]).all()
                assert not torch.isfinite(got[2]).all()
            # the same of the losses: every expert that is left, in every row
            load = torch.bincount(idx.flatten(), minlength=N + 1).int()
            load[N] = T
            for bad in ((float("nan"), 0.0), (0.0, float("nan")), (float("inf"), 0.1)):
                got = B().bfmoe_route_backward(t.cuda(), idx, sc, dgates=torch.randn(T, k, device="cuda"), load=load,
                                               dloss=torch.tensor(bad, device="cuda")).cpu()
                assert (got[:, : N - 3] == 0).all(), (score, renorm, bad)
                assert not torch.isfinite(got[:, N - 3:]).any()


@pytest.mark.parametrize("N", [12, 250, 1024, 1300])
def test_backward_of_masked_choices(N):
    """Chosen experts that a logit or the bias masks have no gate: no gradient from it, whatever theirs is
    (NaN included), and none of the others' gradient passes through them."""
    T, k = 9, 4
    t, _ = make_logits(T, N, "f32", N + 3)
    t[:, : N - 3] = float("-inf")           # three experts are left, one of them masked by the bias
    l = t.double().numpy()
    bias = np.zeros(N, np.float32)
    bias[N - 2] = -np.inf
    db = torch.from_numpy(bias).cuda()
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            sc = scoring(score, renorm=renorm)
            idx, gates = B().bfmoe_route(t.cuda(), k, sc, balance_bias=db, buckets=False)[:2]
            ref, g = S.route(l, k, bias=bias, score=score, renorm=renorm)
            assert np.array_equal(idx.cpu().numpy(), ref)
            off = (torch.from_numpy(g) == 0).cuda()
            assert int(off.sum()) == 2 * T
            dg = torch.randn(T, k, device="cuda")
            dg[off] = float("nan")
            got = B().bfmoe_route_backward(t.cuda(), idx, sc, dgates=dg, balance_bias=db).double().cpu().numpy()
            want, bound = S.route_backward(l, ref, dgates=dg.cpu().numpy(), score=score, renorm=renorm, bias=bias)
            assert np.isfinite(got).all()
            assert (np.abs(got - want) <= half_steps(l) * bound + TINY).all()


def test_two_streams_at_once():
    """Calls that overlap on two streams, each with its workspace, and calls on a stream that is not current,
    whose workspace the binding makes."""
    T, N, k = 4000, 256, 8
    sc = scoring("sigmoid", groups=8, top_groups=4, group_score="top2")
    xs = [make_logits(T, N, "f32", s)[0].cuda() for s in (1, 2)]
    want = [B().bfmoe_route(x, k, sc) for x in xs]
    losses = [B().bfmoe_balance_loss(x, w[0], "sigmoid") for x, w in zip(xs, want)]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [B().bfmoe_route(x, k, sc, stream=s) for x, s in zip(xs, streams)]
        more = [B().bfmoe_balance_loss(x, g[0], "sigmoid", stream=s) for x, g, s in zip(xs, got, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got + more, want + losses):
            for p, q in zip(a, b):
                assert torch.equal(p, q)


def test_backward_repeated_and_foreign_indices():
    """The same expert twice adds up; an index out of range is reported and skipped."""
    t, l = make_logits(9, 40, "f32", 3)
    idx = np.tile(np.array([[3, 3, 7]]), (9, 1))
    for score, renorm in (("sigmoid", False), ("softmax", False)):
        check_backward(t, l, 3, score, renorm, 1.0, aux=False, idx=idx)
    bad = idx.copy()
    bad[4, 1] = 40
    bad[5, 0] = -1
    di = torch.from_numpy(bad.astype(np.int32)).cuda()
    got = B().bfmoe_route_backward(t.cuda(), di, scoring("sigmoid"), dgates=torch.ones(9, 3, device="cuda"))
    assert torch.isfinite(got).all()
    with pytest.raises(B().BfmoeError) as e:
        B().bfmoe_check_device_error()
    assert e.value.status == 7
    B().bfmoe_check_device_error()
    B().bfmoe_balance_loss(t.cuda(), di)
    with pytest.raises(B().BfmoeError):
        B().bfmoe_check_device_error()


# -------------------------------------------------------------------------------------------------------------------
# losses
# -------------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,k", SHAPES + [(3000, 64, 2), (1500, 256, 8)])
def test_balance_loss(T, N, k, dtype):
    t, l = make_logits(T, N, dtype, T + N + 9)
    if T > 6 and N > 2:
        t[1] = float("-inf")
        t[2, : N // 2] = float("-inf")
        t[3, 0] = float("nan")
        t[T - 1] = float("nan")
        t[4] = -300.0
        l = t.double().numpy()
    for score in ("softmax", "sigmoid"):
        idx, _ = S.route(l, k, score=score)
        loss, load = B().bfmoe_balance_loss(t.cuda(), torch.from_numpy(idx.astype(np.int32)).cuda(), score)
        (bal, z), ref, rows = S.balance_loss(l, idx, score)
        assert np.array_equal(load.cpu().numpy(), np.append(ref, rows))
        got = loss.cpu().numpy().astype(np.float64)
        # positive terms only: relative errors do not grow in the sums; lse^2 doubles them
        assert abs(got[0] - bal) <= half_steps(l) * bal
        # lse = max + log(sum): off by half steps of the larger of |max| and 1, absolutely
        assert abs(got[1] - z) <= 2 * half_steps(l) * (z + np.sqrt(z))
    B().bfmoe_check_device_error()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,N", [(1, 200), (1, 104), (5, 128), (37, 256)])
def test_results_do_not_depend_on_earlier_calls(T, N, dtype):
    """Where a warp's rows reach behind the last one, what shared memory held before takes no part."""
    t, _ = make_logits(T, N, dtype, T + N)
    x = t.cuda()
    idx = torch.topk(x.float(), 2)[1].int()
    dg = torch.randn(T, 2, device="cuda")
    dl = torch.tensor([0.3, 0.2], device="cuda")
    sc = scoring("sigmoid")
    first = None
    for before in (0.0, 100.0, float("nan"), -60.0, 3.0):
        big = torch.full((20000, N), before, dtype=x.dtype, device="cuda")
        some = torch.zeros(20000, 2, dtype=torch.int32, device="cuda")
        B().bfmoe_balance_loss(big, some, "sigmoid")
        loss, load = B().bfmoe_balance_loss(x, idx, "sigmoid")
        B().bfmoe_route_backward(big, some, sc, load=load, dloss=dl)
        d = B().bfmoe_route_backward(x, idx, sc, dgates=dg, load=load, dloss=dl)
        if first is None:
            first = loss, d
        assert torch.equal(loss, first[0]) and torch.equal(d, first[1]), before


def test_load_of_two_halves_adds_up():
    """Two ranks' loads added up and a loss gradient each: the gradient of the whole batch."""
    T, N, k = 300, 64, 2
    t, l = make_logits(T, N, "f32", 2)
    idx, _ = S.route(l, k)
    di = torch.from_numpy(idx.astype(np.int32)).cuda()
    x = t.cuda()
    dl = torch.tensor([0.5, 0.1], device="cuda")
    _, whole = B().bfmoe_balance_loss(x, di)
    parts = [B().bfmoe_balance_loss(x[s], di[s])[1] for s in (slice(0, 130), slice(130, T))]
    assert torch.equal(parts[0] + parts[1], whole)
    a = B().bfmoe_route_backward(x, di, scoring(), load=whole, dloss=dl)
    b = torch.cat([B().bfmoe_route_backward(x[s], di[s], scoring(), load=whole, dloss=dl)
                   for s in (slice(0, 130), slice(130, T))])
    assert torch.equal(a, b)


# -------------------------------------------------------------------------------------------------------------------
# refusals of the binding
# -------------------------------------------------------------------------------------------------------------------
def test_binding_refuses():
    m = B()
    x = torch.zeros(4, 8, device="cuda")
    idx = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    sc = scoring()
    for bad in (x.cpu(), x.half(), x.t(), x[0], x.expand(4, 8)[:1].expand(4, 8)):
        with pytest.raises(ValueError):
            m.bfmoe_route(bad, 2, sc)
    with pytest.raises(ValueError):
        m.bfmoe_route(x, 2, sc, balance_bias=torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError):
        m.bfmoe_route_backward(x, idx.long(), sc, dgates=torch.zeros(4, 2, device="cuda"))
    with pytest.raises(ValueError):
        m.bfmoe_route_backward(x, idx, sc, dgates=torch.zeros(4, 2, device="cuda"), dlogits=x.bfloat16())
    with pytest.raises(m.BfmoeError):
        m.bfmoe_route_backward(x, idx, sc, load=torch.zeros(9, dtype=torch.int32, device="cuda"))
    with pytest.raises(m.BfmoeError):
        m.bfmoe_route(x, 9, sc)
    with pytest.raises(m.BfmoeError):
        m.bfmoe_route(x, 2, scoring(groups=3))
    with pytest.raises(ValueError):
        m.Scoring(score="tanh")
