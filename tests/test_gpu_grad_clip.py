"""Global gradient norm and clipping against an exact sum (math.fsum in the
oracle).  Squares and sums are float64, so the norm is off by its own rounding
to float32 (half a step) and a part in 1e13; a scaled gradient by the rounding
of the factor, of the product and, in bfloat16, of the result: two half steps
of float32 plus half a step of the type."""
import numpy as np
import pytest

from oracle import scored_oracle as S

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import ternary_butterfly_experts_b200.build as b
    b.build()


def B():
    import ternary_butterfly_experts_b200 as m
    return m


def host(ts):
    return [t.double().cpu().numpy() for t in ts]


def tensors(sizes, dtype=torch.float32, scale=1.0, offset=0, seed=0):
    """Views of one buffer, each starting where the one before ended (+ offset)."""
    g = torch.Generator().manual_seed(seed)
    n = offset + sum(sizes) + len(sizes)
    buf = (torch.randn(n, generator=g) * scale).to(dtype).cuda()
    out, at = [], offset
    for s in sizes:
        out.append(buf[at:at + s])
        at += s
    return buf, out


SIZES = [[1], [0, 5, 0], [31, 1, 2, 3, 4], [4096], [8191, 8192, 8193], [3, 70001, 16384, 5], [1000] * 40,
         [1 << 20, 7, (1 << 20) + 3]]


@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "x".join(map(str, s[:4])))
def test_norm_and_clip(sizes, dtype, offset):
    buf, gs = tensors(sizes, dtype, 0.03, offset, len(sizes))
    before = buf.clone()
    ref = S.grad_norm(host(gs))
    norm = B().bfmoe_grad_norm(gs)
    assert norm.dtype == torch.float32 and abs(float(norm) - ref) <= (2.0 ** -24 + 1e-13) * ref
    # below the limit: untouched
    assert torch.equal(B().bfmoe_grad_clip(gs, 1.001 * ref + 1e-30), norm)
    assert torch.equal(buf, before)
    # above it: everything times limit / norm, and nothing outside the tensors
    limit = float(np.float32(0.31 * ref))
    want = host(gs)
    assert torch.equal(B().bfmoe_grad_clip(gs, limit), norm)
    for g, w in zip(gs, want):
        w = w * (limit / ref)
        tol = 2 * 2.0 ** -24 + (HALF[dtype] if dtype == torch.bfloat16 else 0) + 1e-12
        assert (np.abs(g.double().cpu().numpy() - w) <= tol * np.abs(w)).all()
    after = buf.clone()
    for g, o in zip(gs, [before[g.storage_offset():g.storage_offset() + g.numel()] for g in gs]):
        after[g.storage_offset():g.storage_offset() + g.numel()] = o
    assert torch.equal(after, before)


def test_out_of_place_and_types():
    _, gs = tensors([5000, 33, 1, 129], torch.float32, 1e-3, 1)
    _, hs = tensors([2000, 17], torch.bfloat16, 1e-3, 1, 5)
    grads = gs + hs
    outs = [torch.full_like(g, 9.0) for g in gs[:2]] + [g.bfloat16() for g in gs[2:]] + [h.float() for h in hs]
    keep = [g.clone() for g in grads]
    ref = S.grad_norm(host(grads))
    lst = B().GradList(grads, out=outs)
    for limit in (0.5 * ref, 2 * ref):   # out is written either way
        by = min(1.0, float(np.float32(limit)) / ref)
        for o in outs:
            o.fill_(9.0)
        B().bfmoe_grad_clip(lst, limit)
        for g, k, o in zip(grads, keep, outs):
            assert torch.equal(g, k)
            w = k.double().cpu().numpy() * by
            tol = 2 * 2.0 ** -24 + HALF[o.dtype] + 1e-12
            assert (np.abs(o.double().cpu().numpy() - w) <= tol * np.abs(w)).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("value", [1e30, 1e-30, 3e38, 1e-40])
def test_range(value, dtype):
    """Squares far outside float32 (1e60, 1e-60): the norm holds."""
    g = torch.full((1000,), value, device="cuda").to(dtype)
    g[3::7] *= -1
    value = float(g[0])
    ref = S.grad_norm(host([g]))
    norm = float(B().bfmoe_grad_norm([g]))
    if ref < 3.4e38:
        assert abs(norm - ref) <= 2.0 ** -24 * ref + 2.0 ** -149
    else:
        assert norm == float("inf")
    if 1e-37 < value:
        B().bfmoe_grad_clip([g], 1.0)
        if ref > 1:
            assert abs(S.grad_norm(host([g])) - 1) <= 2 * 2.0 ** -24 + HALF[dtype]
        else:
            assert (g.abs() == value).all()


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norm_that_is_not_finite_scales_nothing(bad, dtype):
    buf, gs = tensors([5000, 70], dtype, seed=3)
    gs[1][23] = bad
    before = buf.clone()
    norm = B().bfmoe_grad_clip(gs, 0.1)
    assert torch.isnan(norm).all() if bad != bad else (norm == float("inf")).all()
    assert torch.equal(torch.nan_to_num(buf), torch.nan_to_num(before))
    outs = [torch.zeros_like(g) for g in gs]
    B().bfmoe_grad_clip(B().GradList(gs, out=outs), 0.1)
    for g, o in zip(gs, outs):
        assert torch.equal(torch.nan_to_num(g), torch.nan_to_num(o))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norm_beyond_float32_is_inf_and_scales(dtype):
    """The norm of finite gradients that float32 cannot hold: written as inf, the factor from float64."""
    g = torch.tensor([3e38, -3e38, 1.5e38, 1e30], device="cuda").to(dtype)
    want = g.double().cpu().numpy()
    ref = S.grad_norm([want])
    assert ref > 3.5e38
    assert float(B().bfmoe_grad_clip([g], 2.0)) == float("inf")
    want = want * (2.0 / ref)
    tol = 2 * 2.0 ** -24 + HALF[dtype] + 1e-12
    assert (np.abs(g.double().cpu().numpy() - want) <= tol * np.abs(want)).all()


def test_zero_gradients_and_limits():
    g = torch.zeros(100, device="cuda")
    assert float(B().bfmoe_grad_clip([g], 0.0)) == 0.0 and (g == 0).all()
    h = torch.ones(100, device="cuda")
    assert float(B().bfmoe_grad_clip([h], 0.0)) == 10.0 and (h == 0).all()
    h.fill_(2)
    B().bfmoe_grad_clip([h], float("inf"))
    assert (h == 2).all()
    assert float(B().bfmoe_grad_norm([])) == 0.0 and float(B().bfmoe_grad_clip([], 1.0)) == 0.0
    assert float(B().bfmoe_grad_norm([h[:0]])) == 0.0


def test_many_tensors():
    """More tensors than one launch takes."""
    sizes = [(7 * i) % 61 for i in range(1300)]
    buf, gs = tensors(sizes, seed=4)
    ref = S.grad_norm(host(gs))
    want = [w / ref for w in host(gs)]
    assert abs(float(B().bfmoe_grad_clip(gs, 1.0)) - ref) <= (2.0 ** -24 + 1e-13) * ref
    for g, w in zip(gs, want):
        assert (np.abs(g.double().cpu().numpy() - w) <= 2.5 * 2.0 ** -24 * np.abs(w)).all()


def test_more_than_32_bits_of_elements():
    n = (1 << 31) + 4099
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-3:] = 3.0
    g[0] = 4.0
    g[1 << 31] = 2.0
    norm = B().bfmoe_grad_clip([g], 1.0)
    ref = (27 + 16 + 4) ** 0.5
    assert abs(float(norm) - ref) <= 2.0 ** -23 * ref
    for i, v in ((0, 4.0), (1 << 31, 2.0), (n - 1, 3.0)):
        assert abs(float(g[i]) - v / ref) <= 2.0 ** -7 * v / ref
    assert int((g != 0).sum()) == 5


def test_same_result_every_time_and_in_graphs():
    buf, gs = tensors([300000, 17, 4096, 90001], seed=8)
    outs = [torch.empty_like(g) for g in gs]
    lst = B().GradList(gs, out=outs)
    a = B().bfmoe_grad_clip(lst, 1.0)
    first = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        b = B().bfmoe_grad_clip(lst, 1.0)
    for o in outs:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    for o, f in zip(outs, first):
        assert torch.equal(o, f)
    buf.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert abs(float(b) / float(a) - 2) < 1e-6


def test_overlapping_tensors_are_refused():
    m = B()
    buf = torch.ones(100, device="cuda")
    with pytest.raises(m.BfmoeError):
        m.bfmoe_grad_clip([buf, buf], 1.0)
    with pytest.raises(m.BfmoeError):
        m.bfmoe_grad_clip([buf[:60], buf[59:]], 1.0)
    out = torch.empty(100, device="cuda")
    with pytest.raises(m.BfmoeError):
        m.bfmoe_grad_clip(m.GradList([buf[:50], buf[50:]], out=[out[:50], out[49:99]]), 1.0)
    with pytest.raises(m.BfmoeError):
        m.bfmoe_grad_clip(m.GradList([buf[:50]], out=[buf[10:60]]), 1.0)
    # read only: the same tensor twice counts twice
    assert abs(float(m.bfmoe_grad_norm([buf, buf])) - 200 ** 0.5) < 1e-5
    m.bfmoe_grad_clip(m.GradList([buf, buf], out=[out, torch.empty_like(out)]), 1.0)
    assert (buf == 1).all()


def test_binding_refuses():
    m = B()
    g = torch.ones(4, 6, device="cuda")
    for bad in (g.cpu(), g.half(), g.t(), g[:, :3]):
        with pytest.raises(ValueError):
            m.bfmoe_grad_norm([bad])
    with pytest.raises(ValueError):
        m.GradList([g], out=[g, g])
    with pytest.raises(ValueError):
        m.GradList([g], out=[torch.empty(3, device="cuda")])
    for limit in (-1.0, float("nan")):
        with pytest.raises(m.BfmoeError):
            m.bfmoe_grad_clip([g], limit)
