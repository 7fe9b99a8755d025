"""Whose memory the layer objects and the 8-bit calls use: the stream, the graph and the device that a
call runs on, checked on the host with stand-ins for PyTorch's streams, and on
the GPU with a current stream that is busy."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

gpu = pytest.mark.gpu
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    from token_dispatch_grouped_moe_gb300 import build, lib as L
    build.build()
    L.load()
    return L


def fake_stream(handle):
    return SimpleNamespace(cuda_stream=handle, device=torch.device("cpu"))


@pytest.fixture
def streams(monkeypatch):
    """Stand-ins for PyTorch's current stream: ``now()`` is the handle of the
    stream whose memory an allocation takes."""
    state = SimpleNamespace(stack=[fake_stream(1)])
    state.now = lambda: state.stack[-1].cuda_stream

    @contextlib.contextmanager
    def on(s):
        state.stack.append(s if s is not None else state.stack[-1])
        try:
            yield
        finally:
            state.stack.pop()

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: state.stack[-1])
    return state


def host_layer(cls, H=64, F=64, E=8, k=2):
    """A layer object without its weights' memory: its host logic alone."""
    layer = object.__new__(cls)
    t = torch.zeros
    with_init = {"Wg": t(H, E), "W1": t(E, H, F), "W3": t(E, H, F), "W2": t(E, F, H)}
    return layer, with_init, k


def fp8_host_layer(lib, monkeypatch):
    layer, w, k = host_layer(lib.MoEFp8Layer)
    monkeypatch.setattr(lib.Fp8Weights, "from_bf16", classmethod(lambda cls, *a, **kw: None))
    layer.__init__(None, w["Wg"], w["W1"], w["W3"], w["W2"], k)
    return layer


def record_workspaces(lib, monkeypatch, streams, name):
    """The stream that each new workspace was made on."""
    made = []

    def workspace(dims=None, device=None):
        made.append(streams.now())
        return torch.zeros(16, dtype=torch.uint8)

    monkeypatch.setattr(lib, name, workspace)
    return made


def test_fp8_layer_workspace_is_made_on_the_calls_stream(lib, monkeypatch, streams):
    made = record_workspaces(lib, monkeypatch, streams, "fp8_workspace")
    layer = fp8_host_layer(lib, monkeypatch)
    used = []
    monkeypatch.setattr(lib, "add_rmsnorm_fp8", lambda *a, **kw: (None,) * 4)
    monkeypatch.setattr(lib, "fp8_layer_forward", lambda dims, y, q, s, Wg, f, ws, **kw: used.append(ws))
    x, side = torch.zeros(4, 64), fake_stream(2)
    layer.forward(x, stream=side)
    assert made == [2]
    layer.forward(x, stream=side)
    assert made == [2] and used[0] is used[1]
    # another stream has a workspace of its own, and the first keeps its
    layer.forward(x)
    assert made == [2, 1] and used[2] is not used[0]
    layer.forward(x, stream=side)
    assert made == [2, 1] and used[3] is used[0]
    # more rows: again on the call's stream
    layer.forward(torch.zeros(9, 64), stream=side)
    assert made == [2, 1, 2]


def test_bf16_layer_workspace_is_made_on_the_calls_stream(lib, monkeypatch, streams):
    made = record_workspaces(lib, monkeypatch, streams, "workspace")
    layer, w, k = host_layer(lib.MoELayer)
    layer.__init__(w["Wg"], w["W1"], w["W3"], w["W2"], k)
    used = []
    monkeypatch.setattr(lib, "layer_forward", lambda dims, x, Wg, W1, W3, W2, ws, *a, **kw: used.append(ws))
    x, side = torch.zeros(4, 64), fake_stream(2)
    layer.forward(x, stream=side)
    layer.forward(x)
    layer.forward(x, stream=side)
    assert made == [2, 1] and used[0] is used[2] and used[1] is not used[0]
    layer.forward(torch.zeros(9, 64), stream=side)
    assert made == [2, 1, 2]


# ------------------------------------------------------------------ on the GPU

def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def weights(g, H, F, E):
    rnd = lambda *s, sigma=0.05: (torch.randn(*s, generator=g, device="cuda") * sigma).bfloat16()  # noqa: E731
    return rnd(H, E), rnd(E, H, F), rnd(E, H, F), rnd(E, F, H)


def late_fill(sizes, value):
    """Blocks of these sizes, on the current stream: freed by the host at once,
    filled by the stream only after a while. Memory of this stream's pool that a
    call on another stream takes now is overwritten by that fill."""
    torch.cuda._sleep(20_000_000)
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    for b in blocks:
        b.fill_(value)


@gpu
def test_fp8_layer_on_a_side_stream_while_the_current_one_is_busy(lib):
    """A fresh layer's first calls, of several lengths, on a side stream: the
    workspaces are not memory that the current stream still writes, nor zeroed
    by it behind the layer's back."""
    g = gen(1)
    H, F, E, k = 512, 256, 8, 2
    Wg, W1, W3, W2 = weights(g, H, F, E)
    calls = [torch.randn(T, H, generator=g, device="cuda").bfloat16() for T in (1, 37, 5, 300)]
    want = [lib.MoEFp8Layer(None, Wg, W1, W3, W2, k).forward(x)[0] for x in calls]
    layer = lib.MoEFp8Layer(None, Wg, W1, W3, W2, k)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for x, w in zip(calls, want):
        size = lib.fp8_workspace_size(layer.dims(x.shape[0]))
        late_fill([size], 0xFF)
        got, _ = layer.forward(x, stream=side)
        with torch.cuda.stream(side):
            assert torch.equal(got, w)   # before the current stream's fills
        torch.cuda.synchronize()
        assert torch.equal(got, w)       # and behind them
        assert lib.check(layer.workspace(x.shape[0], side)) == lib.MOE_OK


@gpu
def test_bf16_layer_on_a_side_stream_while_the_current_one_is_busy(lib):
    g = gen(2)
    H, F, E, k = 512, 256, 8, 2
    Wg, W1, W3, W2 = weights(g, H, F, E)
    calls = [torch.randn(T, H, generator=g, device="cuda").bfloat16() for T in (1, 37, 5, 300)]
    want = [lib.MoELayer(Wg, W1, W3, W2, k).forward(x) for x in calls]
    layer = lib.MoELayer(Wg, W1, W3, W2, k)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for x, w in zip(calls, want):
        out = torch.empty_like(w)
        late_fill([lib.workspace_size(layer.dims(x.shape[0]))], 0xFF)
        layer.forward(x, out=out, stream=side)
        with torch.cuda.stream(side):
            assert torch.equal(out, w)
        torch.cuda.synchronize()
        assert torch.equal(out, w)
        assert lib.check(layer.workspace(x.shape[0], side)) == lib.MOE_OK
