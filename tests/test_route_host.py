"""Host-side checks of the routing, loss and gradient-clipping entry points:
refused before any launch, on a machine without a GPU."""
import ctypes

import pytest

from ternary_butterfly_experts_b200 import build, capi


@pytest.fixture(scope="module")
def L():
    build.build()
    return capi.lib()


def sc(score=0, groups=1, top=1, gs=0, renorm=1, scale=1.0):
    return ctypes.byref(capi.BfmoeScoring(score, groups, top, gs, renorm, scale))


F32, BF16, EINVAL, EUNS, EWS, OK = capi.BFMOE_F32, capi.BFMOE_BF16, 1, 3, 4, 0
WS = (256, 1 << 30)


def route(L, logits=64, dtype=F32, T=4, ld=8, N=8, k=2, s=None, bias=None, idx=64, gates=64, counts=64, offsets=64,
          rows=64, ws=WS):
    return L.bfmoe_route(logits, dtype, T, ld, N, k, s if s is not None else sc(), bias, idx, gates, counts, offsets,
                         rows, ws[0], ws[1], None)


def test_route_refuses(L):
    n0 = L.bfmoe_launch_count()
    for kw in (dict(k=0), dict(k=9, N=16, ld=16), dict(k=3, N=2, ld=2), dict(N=0), dict(N=4097, ld=4097), dict(T=-1),
               dict(ld=7), dict(dtype=2), dict(s=sc(score=2)), dict(s=sc(gs=5)), dict(s=sc(groups=3)),
               dict(s=sc(groups=0)), dict(N=130, ld=130, s=sc(groups=65)), dict(s=sc(groups=4, top=0)),
               dict(s=sc(groups=4, top=5)), dict(s=sc(groups=8, top=1)), dict(s=sc(scale=float("nan"))),
               dict(s=sc(scale=float("inf"))), dict(logits=None), dict(idx=None), dict(gates=None), dict(counts=None),
               dict(offsets=None), dict(rows=None), dict(logits=66), dict(logits=65, dtype=BF16)):
        assert route(L, **kw) == EINVAL, kw
    assert L.bfmoe_route(64, F32, 4, 8, 8, 2, None, None, 64, 64, 64, 64, 64, 256, 1 << 30, None) == EINVAL
    assert route(L, T=1 << 30, k=8) == EUNS
    assert route(L, T=0x7ff00001, k=1) == EUNS
    for ws in ((None, 0), (256, 16), (264, 1 << 30)):
        assert route(L, ws=ws) == EWS
    # no tokens and no buckets: nothing to do
    assert route(L, T=0, logits=None, idx=None, gates=None, counts=None, offsets=None, rows=None) == OK
    assert L.bfmoe_launch_count() == n0


def test_balance_loss_refuses(L):
    n0 = L.bfmoe_launch_count()
    f = L.bfmoe_balance_loss
    assert f(64, F32, 4, 8, 8, 2, 3, 64, 64, 64, *WS, None) == EINVAL
    assert f(None, F32, 4, 8, 8, 2, 0, 64, 64, 64, *WS, None) == EINVAL
    assert f(64, F32, 4, 8, 8, 2, 0, None, 64, 64, *WS, None) == EINVAL
    assert f(64, F32, 4, 8, 8, 2, 0, 64, None, 64, *WS, None) == EINVAL
    assert f(64, F32, 4, 8, 8, 2, 0, 64, 64, None, *WS, None) == EINVAL
    assert f(64, F32, 4, 7, 8, 2, 0, 64, 64, 64, *WS, None) == EINVAL
    assert f(64, 7, 4, 8, 8, 2, 0, 64, 64, 64, *WS, None) == EINVAL
    assert f(64, F32, 4, 8, 8, 2, 0, 64, 64, 64, None, 0, None) == EWS
    assert f(64, F32, 4, 8, 8, 2, 0, 64, 64, 64, 256, 8, None) == EWS
    assert L.bfmoe_launch_count() == n0


def test_route_backward_refuses(L):
    n0 = L.bfmoe_launch_count()

    def f(logits=64, dtype=F32, T=4, ld=8, N=8, k=2, s=None, idx=64, dg=64, load=64, dloss=64, out=64, ldd=8):
        return L.bfmoe_route_backward(logits, dtype, T, ld, N, k, s if s is not None else sc(), None, idx, dg, load,
                                      dloss, out, ldd, None)

    for kw in (dict(ldd=7), dict(load=None), dict(dloss=None), dict(logits=None), dict(out=None), dict(idx=None),
               dict(out=66), dict(ld=10, ldd=8), dict(s=sc(score=9)), dict(k=0), dict(dtype=4)):
        assert f(**kw) == EINVAL, kw
    assert f(T=0, logits=None, out=None, idx=None) == OK
    assert L.bfmoe_launch_count() == n0


def test_route_workspace_size(L):
    assert L.bfmoe_route_workspace_size(256, 16384, 8) % 256 == 0
    assert L.bfmoe_route_workspace_size(256, 16384, 8) >= 16384 // 128 * 256 * 4
    for bad in ((0, 4, 1), (8, -1, 1), (8, 4, 9), (4097, 4, 1)):
        assert L.bfmoe_route_workspace_size(*bad) == 0
    assert L.bfmoe_route_workspace_size(8, 0, 1) > 0


def test_router_logits_and_expert_backward_refuse(L):
    n0 = L.bfmoe_launch_count()
    f = L.bfmoe_router_logits
    assert f(64, BF16, 4, 63, 64, None, 8, 64, *WS, None) == EINVAL
    assert f(None, BF16, 4, 64, 64, None, 8, 64, *WS, None) == EINVAL
    assert f(64, BF16, 4, 64, 64, None, 8, 80, *WS, None) == EINVAL       # logits not 32-byte aligned
    assert f(64, BF16, 4, 64, 64, None, 8, 64, None, 0, None) == EWS
    assert f(None, BF16, 0, 64, 64, None, 8, None, None, 0, None) == OK
    lay = capi.BfmoeLayer(64, 4, 16, ctypes.c_float(0.1), 16, 16)
    g = L.bfmoe_expert_backward
    args = [16, BF16, 4, 2, 16, 16, 16, 16, 16, 16, 16, 16, 16, 16, 16]
    assert g(None, *args, *WS, None) == EINVAL
    for i in (0, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14):
        bad = list(args)
        bad[i] = None
        assert g(ctypes.byref(lay), *bad, *WS, None) == EINVAL, i
    assert g(ctypes.byref(lay), *args, None, 0, None) == EWS
    assert L.bfmoe_launch_count() == n0


def grads(*items):
    a = (capi.BfmoeGrad * max(len(items), 1))()
    for i, it in enumerate(items):
        a[i] = capi.BfmoeGrad(*it)
    return a, len(items)


def test_grad_calls_refuse(L):
    n0 = L.bfmoe_launch_count()
    good = (4096, None, 10, F32, F32)
    for fn, extra in ((L.bfmoe_grad_norm, ()), (L.bfmoe_grad_clip, (1.0,))):
        assert fn(None, 1, *extra, 64, *WS, None) == EINVAL
        assert fn(*grads(good)[:1], -1, *extra, 64, *WS, None) == EINVAL
        assert fn(*grads(good), *extra, None, *WS, None) == EINVAL
        for bad in ((None, None, 10, F32, F32), (4096, None, -1, F32, F32), (4096, None, 10, 5, F32),
                    (4098, None, 10, F32, F32), (4097, None, 10, BF16, F32)):
            assert fn(*grads(good, bad), *extra, 64, *WS, None) == EINVAL, bad
        assert fn(*grads(good), *extra, 64, None, 0, None) == EWS
        assert fn(*grads(good), *extra, 64, 256, 8, None) == EWS
        assert fn(*grads((4096, None, (1 << 62) - 1, F32, F32)), *extra, 64, *WS, None) in (EINVAL, EUNS)
    c = L.bfmoe_grad_clip
    assert c(*grads(good), -1.0, 64, *WS, None) == EINVAL
    assert c(*grads(good), float("nan"), 64, *WS, None) == EINVAL
    for bad in ([good, good],                                                      # the same tensor twice
                [good, (4096 + 36, None, 5, F32, F32)],                            # the last element shared
                [(4096, 8192, 10, F32, F32), (5000, 8192 + 36, 10, F32, F32)],     # outputs overlap
                [(4096, 4096, 10, F32, BF16)],                                     # in place into another type
                [(4096, 4100, 10, F32, F32)],                                      # output over its own input, shifted
                [(4096, 8192, 10, F32, F32), (8192, 12288, 10, F32, F32)],         # output over another's input
                [(4096, 8191, 10, F32, F32)], [(4096, 8192, 10, F32, 3)]):
        assert c(*grads(*bad), 1.0, 64, *WS, None) == EINVAL, bad
    assert L.bfmoe_launch_count() == n0


def test_a_changed_scoring_is_what_calls_see():
    import ternary_butterfly_experts_b200 as B

    sc = B.Scoring("sigmoid", n_groups=8, top_groups=4, group_score="top2", scale=2.5)
    assert repr(sc) == ("Scoring(score='sigmoid', n_groups=8, top_groups=4, group_score='top2', renormalize=True, "
                        "scale=2.5)")
    new = dict(score="softmax", n_groups=4, top_groups=2, group_score="max", renormalize=False, scale=0.3)
    for name, value in new.items():
        setattr(sc, name, value)
        assert getattr(sc, name) == value
    c = ctypes.cast(sc.ref, ctypes.POINTER(capi.BfmoeScoring)).contents
    assert (c.score, c.n_groups, c.top_groups, c.group_score, c.renormalize) == (0, 4, 2, 0, 0)
    assert c.scale == ctypes.c_float(0.3).value
    assert repr(sc) == repr(B.Scoring(**new))
    for name, value in (("score", "tanh"), ("group_score", "sum")):
        with pytest.raises(ValueError):
            setattr(sc, name, value)
        with pytest.raises(ValueError):
            B.Scoring(**{name: value})
    assert (sc.score, sc.group_score) == ("softmax", "max")
