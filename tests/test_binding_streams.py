"""Where the binding makes the outputs and the scratch of a call with
``stream=``: in that stream's memory pool.  (A block of the current stream's
pool may have been freed with kernels still queued there that write it; the
call on the other stream is not ordered behind them.)  The allocator is
watched on the CPU, the library is a stand-in."""
import contextlib

import pytest

torch = pytest.importorskip("torch")
from torch.overrides import TorchFunctionMode

import ternary_butterfly_experts_b200 as B

MAKERS = {torch.empty, torch.empty_like, torch.zeros, torch.Tensor.new_empty}


class Dev(torch.Tensor):
    """A CPU tensor that says it is on CUDA device 0."""
    is_cuda = property(lambda self: True)

    kept = []  # (address, stream) of record_stream

    def get_device(self):
        return 0

    def record_stream(self, s):
        Dev.kept.append((self.data_ptr(), s))


class Watch(TorchFunctionMode):
    def __init__(self):
        super().__init__()
        self.stream, self.made = None, []

    def __torch_function__(self, func, types, args=(), kwargs=None):
        kwargs = dict(kwargs or {})
        if func not in MAKERS:
            return func(*args, **kwargs)
        if func is torch.empty:
            kwargs["device"] = "cpu"
        t = func(*args, **kwargs).as_subclass(Dev)
        self.made.append((t, self.stream))
        return t


class Stream:
    cuda_stream = 77


class Lib:
    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        if name.endswith("_size"):
            return lambda *a: 4096

        def call(*a):
            self.streams.append(a[-1])
            return 0
        return call


@pytest.fixture
def watch(monkeypatch):
    w, lib = Watch(), Lib()

    @contextlib.contextmanager
    def stream(s):
        before, w.stream = w.stream, s
        yield
        w.stream = before

    monkeypatch.setattr(Dev, "kept", [])
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: "current")
    monkeypatch.setattr(B, "_stream", lambda s=None: 0 if s is None else s.cuda_stream)
    monkeypatch.setattr(B.capi, "lib", lambda: lib)
    w.lib = lib
    MODE[:] = [w]
    return w


def dev(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Dev)


def i32(*shape):
    return dev(*shape, dtype=torch.int32)


T, N, K, D = 6, 8, 2, 16


def layer():
    return B.Layer(i32(D, 1), 0.5, dev(N, 4, D // 2), dev(N, 4, D // 2))


def routing():
    return i32(T, K), dev(T, K), i32(N), i32(N + 1), i32(T * K)


NEW = {
    "router_logits": lambda **kw: B.bfmoe_router_logits(dev(T, D), dev(N, D), **kw),
    "route": lambda **kw: B.bfmoe_route(dev(T, N), K, B.Scoring(), **kw),
    "route_no_buckets": lambda **kw: B.bfmoe_route(dev(T, N), K, B.Scoring(), buckets=False, **kw),
    "balance_loss": lambda **kw: B.bfmoe_balance_loss(dev(T, N), i32(T, K), **kw),
    "route_backward": lambda **kw: B.bfmoe_route_backward(dev(T, N), i32(T, K), B.Scoring(), dgates=dev(T, K), **kw),
    "expert_backward": lambda **kw: B.bfmoe_expert_backward(layer(), dev(T, D), K, routing(), dev(T, D), **kw),
    "grad_norm": lambda **kw: B.bfmoe_grad_norm([dev(5)], **kw),
    "grad_clip": lambda **kw: B.bfmoe_grad_clip([dev(5)], 1.0, **kw),
}


def prepared(**kw):
    a = layer().prepare(**kw)
    return a.tables


def gate_prepared(**kw):
    a = layer().prepare_gate(dev(N, D), **kw)
    return a.gate_parts


def host_scratch(**kw):
    moe = B.ButterflyMoE(layer(), dev(N, D), None, K, T, torch.float32)
    Dev.kept.clear()
    MODE[0].made.clear()
    moe.forward_host(torch.ones(T, D), torch.ones(T, D), **kw)
    return moe.ws_host


OLD = {
    "pack_base": lambda **kw: B.bfmoe_pack_base(dev(D, D, dtype=torch.int8), **kw),
    "unpack_base": lambda **kw: B.bfmoe_unpack_base(i32(D, 1), D, **kw),
    "router_topk": lambda **kw: B.bfmoe_router_topk(dev(T, D), dev(N, D), None, K, i32(64), **kw),
    "router_topk_no_buckets": lambda **kw: B.bfmoe_router_topk(dev(T, D), dev(N, D), None, K, i32(64), buckets=False, **kw),
    "router_topk_noalloc": lambda **kw: B.bfmoe_router_topk_noalloc(dev(T, D), dev(N, D), None, K, **kw),
    "forward": lambda **kw: B.bfmoe_forward(layer(), dev(T, D), K, *[routing()[i] for i in (0, 1, 3, 4)], i32(64), **kw),
    "decode_forward": lambda **kw: B.bfmoe_decode_forward(layer(), dev(T, D), K, *routing()[:2], **kw),
    "moe_forward": lambda **kw: [t for o in B.bfmoe_moe_forward(layer(), dev(T, D), dev(N, D), None, K, i32(64), **kw)
                                 for t in ([o] if isinstance(o, torch.Tensor) else o)],
    "backward": lambda **kw: B.bfmoe_backward(layer(), dev(T, D), K, dev(N, D), routing(), dev(T, D), **kw),
    "materialize_expert": lambda **kw: B.bfmoe_materialize_expert(layer(), 0, **kw),
    "prepare": prepared,
    "prepare_gate": gate_prepared,
    "forward_host": host_scratch,
}
MODE = []


def tensors(out):
    if isinstance(out, dict):
        out = out.values()
    return [t for t in (out if not isinstance(out, torch.Tensor) else [out]) if t is not None]


def check(watch, call):
    s = Stream()
    with watch:
        out = call(stream=s)
    made = [(t, on) for t, on in watch.made]
    watch.made = []
    assert watch.lib.streams[-1] == 77
    mine = [t for t in tensors(out)]
    for t in mine:
        assert any(t.data_ptr() == m.data_ptr() and on is s for m, on in made), "an output is of another stream's pool"
        assert t.numel() == 0 or (t.data_ptr(), "current") in Dev.kept, "the caller's stream is not known"
    scratch = [(m, on) for m, on in made if m.dtype == torch.uint8]
    assert all(on is s for _, on in scratch), "scratch of another stream's pool"
    # without a stream nothing changes hands
    Dev.kept.clear()
    with watch:
        call()
    assert all(on is None for _, on in watch.made) and not Dev.kept


@pytest.mark.parametrize("name", sorted(NEW))
def test_outputs_and_scratch_belong_to_the_stream_of_the_call(watch, name):
    check(watch, NEW[name])


@pytest.mark.parametrize("name", sorted(OLD))
def test_so_do_those_of_the_layer_calls(watch, name):
    check(watch, OLD[name])


def test_a_kept_list_is_used_on_the_stream_of_the_call(watch):
    with watch:
        g = B.GradList([dev(5)])
        s = Stream()
        watch.made = []
        norm = B.bfmoe_grad_norm(g, stream=s)
    assert (g.ws.data_ptr(), s) in Dev.kept
    assert [on for t, on in watch.made if t.data_ptr() == norm.data_ptr()] == [s]


@pytest.mark.gpu
def test_a_call_beside_a_busy_current_stream():
    """The current stream still has to write blocks that were freed just before the call on another stream."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    T, N, k = 3000, 256, 4
    x = torch.randn(T, N, device="cuda")
    gs = [torch.randn(70001, device="cuda"), torch.randn(513, device="cuda")]
    sc, s = B.Scoring("sigmoid"), torch.cuda.Stream()
    dg, dl = torch.randn(T, k, device="cuda"), torch.tensor([0.1, 0.2], device="cuda")

    def step(stream):
        out = B.bfmoe_route(x, k, sc, stream=stream)
        loss, load = B.bfmoe_balance_loss(x, out[0], "sigmoid", stream=stream)
        d = B.bfmoe_route_backward(x, out[0], sc, dgates=dg, load=load, dloss=dl, stream=stream)
        return (*out, loss, load, d, B.bfmoe_grad_norm(gs, stream=stream))

    want = step(None)
    torch.cuda.synchronize()
    for _ in range(5):
        torch.cuda._sleep(20_000_000)  # about 10 ms
        for n in (1 << 10, 1 << 14, 1 << 18, 1 << 20, 1 << 22, 3000 * 256 * 4):
            many = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(8)]
            for t in many:
                t.fill_(0x7f)
            del many, t
        got = step(s)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    B.bfmoe_check_device_error()
