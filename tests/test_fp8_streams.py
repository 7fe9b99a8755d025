"""Whose memory the layer objects and the 8-bit calls use: the stream, the graph and the device that a
call runs on, checked on the host with stand-ins for PyTorch's streams, and on
the GPU with a current stream that is busy."""
import contextlib
import functools
from types import SimpleNamespace

import pytest
import torch
from torch._subclasses import FakeTensorMode

gpu = pytest.mark.gpu
pytestmark = pytest.mark.filterwarnings("ignore:Accessing the data pointer of FakeTensor")
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    from token_dispatch_grouped_moe_gb300 import build, lib as L
    build.build()
    L.load()
    return L


def fake_stream(handle, device=0):
    return SimpleNamespace(cuda_stream=handle, device=torch.device("cuda", device))


@pytest.fixture
def streams(monkeypatch):
    """Stand-ins for PyTorch's streams and devices: ``now()`` is the handle of the
    stream whose memory an allocation takes, and whose device a launch runs on.
    Tensors are FakeTensors: they have a device and no memory."""
    state = SimpleNamespace(stack=[fake_stream(1)])
    state.now = lambda: state.stack[-1].cuda_stream
    state.device = lambda: state.stack[-1].device.index

    @contextlib.contextmanager
    def on(s):
        state.stack.append(s if s is not None else state.stack[-1])
        try:
            yield
        finally:
            state.stack.pop()

    def device_stream(device=None):
        """The current stream of a device: 1 of device 0, 101 of device 1."""
        index = state.device() if device is None else torch.device(device).index
        return state.stack[-1] if index == state.device() else fake_stream(1 + 100 * index, index)

    monkeypatch.setattr(torch.cuda, "device", lambda d: on(device_stream(d)))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: state.device())
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: device_stream(f"cuda:{index}").cuda_stream)
    state.captured = set()   # handles of streams that are being captured
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state.now() in state.captured)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", device_stream)
    with FakeTensorMode(allow_non_fake_inputs=True):
        yield state


def host_layer(cls, H=64, F=64, E=8, k=2):
    """A layer object without its weights' memory: its host logic alone."""
    layer = object.__new__(cls)
    t = functools.partial(torch.empty, device="cuda:0", dtype=torch.bfloat16)
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


@pytest.mark.parametrize("bits", [8, 16])
def test_layer_workspace_grows_only(lib, monkeypatch, streams, bits):
    """Batches of changing length keep one workspace, large enough for each."""
    made = record_workspaces(lib, monkeypatch, streams, "fp8_workspace" if bits == 8 else "workspace")
    if bits == 8:
        layer = fp8_host_layer(lib, monkeypatch)
    else:
        layer, w, k = host_layer(lib.MoELayer)
        layer.__init__(w["Wg"], w["W1"], w["W3"], w["W2"], k)
    first = layer.workspace(100)
    assert all(layer.workspace(T) is first for T in (1, 64, 100, 0, 7)) and len(made) == 1
    # row by row: a few workspaces, not one for each length
    for T in range(101, 1000):
        layer.workspace(T)
    assert len(made) <= 12


@pytest.mark.parametrize("bits", [8, 16])
def test_layer_workspace_of_a_graph_is_the_graphs(lib, monkeypatch, streams, bits):
    """A captured call neither takes the workspace that is kept for eager calls
    (which is given back once a longer batch has outgrown it, under the graph's
    feet) nor leaves its own for them (whose zeroing runs with the graph only)."""
    made = record_workspaces(lib, monkeypatch, streams, "fp8_workspace" if bits == 8 else "workspace")
    if bits == 8:
        layer = fp8_host_layer(lib, monkeypatch)
    else:
        layer, w, k = host_layer(lib.MoELayer)
        layer.__init__(w["Wg"], w["W1"], w["W3"], w["W2"], k)
    side = fake_stream(2)
    eager = layer.workspace(8, side)
    streams.captured.add(2)
    first, second = layer.workspace(8, side), layer.workspace(8, side)
    assert first is not eager and second is not eager and first is not second and made == [2, 2, 2]
    longer = layer.workspace(16, side)
    streams.captured.clear()
    assert layer.workspace(8, side) is eager
    assert layer.workspace(16, side) is not longer


@pytest.mark.parametrize("H,F,E,k,Fs", [(64, 64, 8, 2, 0), (2048, 1408, 64, 6, 2816), (4096, 14336, 8, 2, 0),
                                        (512, 64, 256, 8, 0), (1024, 512, 128, 8, 64)])
def test_workspace_sizes_grow_with_the_rows(lib, H, F, E, k, Fs):
    """A workspace of more rows is large enough for fewer."""
    rows = [0, 1, 2, 31, 127, 128, 129, 511, 512, 513, 1024, 4095, 4096, 4097, 8192, 32768, 100000]
    for size in (lib.fp8_workspace_size, lib.workspace_size):
        sizes = [size(lib.make_dims(T, H, F, E, k, Fs)) for T in rows]
        assert sizes == sorted(sizes) and sizes[0] > 0


def test_fp8_workspace_zeroes_its_head_only(lib, monkeypatch):
    """The zeros that the calls ask for, not tens of megabytes or gigabytes of them."""
    import re
    header = open(__file__.replace("tests/test_fp8_streams.py", "include/moe.h")).read()
    zeros = int(re.search(r"#define MOE_FP8_WORKSPACE_ZEROS (\d+)", header).group(1))
    assert lib.FP8_WORKSPACE_ZEROS == zeros <= 4096
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: real(*a, **kw).fill_(0xA5))
    for dims in (None, lib.make_dims(5, 64, 64, 8, 2)):
        ws = lib.fp8_workspace(dims, device="cpu")
        assert ws.numel() == lib.fp8_workspace_size(dims)
        assert not ws[:zeros].any() and bool((ws[zeros:] == 0xA5).all())


class FakeLibrary:
    """Answers every call with MOE_OK and computes nothing; keeps each call's
    device and stream (its last argument)."""

    def __init__(self, streams):
        self.streams, self.calls = streams, []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, self.streams.device(), args[-1].value))
            return 0
        return call


def record_allocations(monkeypatch, streams):
    """The stream that each torch.empty was called on."""
    taken, real = [], torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: (taken.append(streams.now()), real(*a, **kw))[1])
    return taken


def test_quantized_weights_are_the_calls_streams_memory(lib, monkeypatch, streams):
    monkeypatch.setattr(lib, "load", lambda: FakeLibrary(streams))
    w = torch.empty(2, 64, 64, dtype=torch.bfloat16, device="cuda:0")
    taken = record_allocations(monkeypatch, streams)
    lib.fp8_quantize_weight(w, stream=fake_stream(2))
    assert taken == [2, 2]
    lib.Fp8Weights.from_bf16(w, w, w, stream=fake_stream(3))
    assert taken[2:] == [3] * 6
    lib.fp8_quantize_weight(w)
    assert taken[8:] == [1, 1]


def fake_fp8_layer_call(lib, device, T=4, H=64, F=64, E=8, **kw):
    t = functools.partial(torch.empty, device=device)
    f = torch.float32
    w = lib.Fp8Weights(t(E, F, H, dtype=FP8), t(E, 1, 1, dtype=f), t(E, F, H, dtype=FP8), t(E, 1, 1, dtype=f),
                       t(E, H, F, dtype=FP8), t(E, 1, 1, dtype=f))
    args = dict(x=t(T, H, dtype=torch.bfloat16), xq=t(T, H, dtype=FP8), xq_scale=t(T, 1, dtype=f),
                Wg=t(H, E, dtype=torch.bfloat16), routed=w, ws=t(1 << 20, dtype=torch.uint8))
    return lib.fp8_layer_forward(lib.make_dims(T, H, F, E, 2), **{**args, **kw})


def test_calls_run_on_their_tensors_device(lib, monkeypatch, streams):
    """Tensors of device 1 while device 0 is the current one."""
    fake = FakeLibrary(streams)
    monkeypatch.setattr(lib, "load", lambda: fake)
    w = torch.empty(2, 64, 64, dtype=torch.bfloat16, device="cuda:1")
    lib.fp8_quantize_weight(w)
    lib.fp8_quantize_weight(w, stream=fake_stream(7, 1))
    fake_fp8_layer_call(lib, "cuda:1")
    fake_fp8_layer_call(lib, "cuda:1", stream=fake_stream(7, 1))
    assert [c[1:] for c in fake.calls] == [(1, 101), (1, 7), (1, 101), (1, 7)]
    fake_fp8_layer_call(lib, "cuda:0")
    assert fake.calls[-1][1:] == (0, 1) and streams.device() == 0
    # the memory that lib.check looks at
    lib.check(torch.empty(256, dtype=torch.uint8, device="cuda:1"))
    assert fake.calls[-1][1:] == (1, 101)
    # a stream of one device cannot order work on another's tensors
    q, scale = torch.empty(4, 64, dtype=FP8, device="cuda:1"), torch.empty(4, 1, device="cuda:1")
    for call in (lambda **kw: lib.fp8_quantize_weight(w, **kw), lambda **kw: fake_fp8_layer_call(lib, "cuda:1", **kw),
                 lambda **kw: lib.add_rmsnorm_fp8(w[0], **kw), lambda **kw: lib.fp8_matmul(q, scale, q, scale, q, **kw),
                 lambda **kw: lib.fp8_gated(q, scale, q, scale, q, scale, q, **kw)):
        with pytest.raises(ValueError, match="stream"):
            call(stream=fake_stream(7, 0))


def test_layer_call_refuses_what_its_kernels_cannot_take(lib, monkeypatch, streams):
    """The workspace and the routing outputs: type, size, layout and device, and
    tensors in host memory, before the library is called."""
    fake = FakeLibrary(streams)
    monkeypatch.setattr(lib, "load", lambda: fake)
    t = functools.partial(torch.empty, device="cuda:0")
    T, E, k = 4, 8, 2

    def routing(**kw):
        good = dict(topk_idx=t(T, k, dtype=torch.int32), topk_w=t(T, k), counts=t(E, dtype=torch.int32),
                    offsets=t(E + 1, dtype=torch.int32), src_row=t(T * k, dtype=torch.int32),
                    inv_pos=t(T * k, dtype=torch.int32))
        return lib.Routing(**{**good, **kw})

    fake_fp8_layer_call(lib, "cuda:0", routing=routing())
    assert len(fake.calls) == 1
    i32 = dict(dtype=torch.int32)
    bad = [dict(ws=t(1 << 18, **i32)), dict(ws=t(1 << 21, dtype=torch.uint8)[::2]),
           dict(ws=torch.empty(1 << 20, dtype=torch.uint8)), dict(ws=t(1 << 20, dtype=torch.uint8).to("cuda:1"))]
    bad += [dict(routing=routing(**kw)) for kw in (
        dict(topk_idx=t(T, k, dtype=torch.int64)), dict(topk_idx=t(T, k + 1, **i32)), dict(topk_w=t(T, k, dtype=torch.bfloat16)),
        dict(counts=t(E - 1, **i32)), dict(offsets=t(E, **i32)), dict(src_row=t(T, **i32)),
        dict(inv_pos=t(2 * T * k, **i32)[::2]), dict(inv_pos=torch.empty(T * k, **i32)))]
    for kw in bad:
        with pytest.raises(ValueError):
            fake_fp8_layer_call(lib, "cuda:0", **kw)
    with pytest.raises(ValueError):
        fake_fp8_layer_call(lib, "cpu")
    with pytest.raises(ValueError):
        lib.fp8_quantize_weight(torch.empty(2, 64, 64, dtype=torch.bfloat16))
    assert len(fake.calls) == 1


def bf16_calls(lib, device, T=4, H=64, F=64, E=8, k=2):
    """Every bf16 call that makes its outputs, on tensors of one device."""
    t = functools.partial(torch.empty, device=device)
    bf, i32 = dict(dtype=torch.bfloat16), dict(dtype=torch.int32)
    d = lib.make_dims(T, H, F, E, k)
    x, Wg, W1, W2 = t(T, H, **bf), t(H, E, **bf), t(E, H, F, **bf), t(E, F, H, **bf)
    idx, ws, slot = t(T, k, **i32), t(1 << 20, dtype=torch.uint8), t(k, T, H)
    return [lambda **kw: lib.route(d, x, Wg, **kw), lambda **kw: lib.permute(d, idx, ws, **kw),
            lambda **kw: lib.permute_static(d, idx, **kw), lambda **kw: lib.combine(d, slot, **kw),
            lambda **kw: lib.expert_ffn(d, x, t(T * k, **i32), t(E + 1, **i32), W1, W1, W2, t(T, k), ws, **kw),
            lambda **kw: lib.layer_forward(d, x, Wg, W1, W1, W2, ws, **kw),
            lambda **kw: lib.route_tc_selftest(d, x, Wg, ws, **kw),
            lambda **kw: lib.layer_forward_host(d, torch.empty(T, H, **bf), Wg, W1, W1, W2, ws, x, x,
                                                torch.empty(T, H, **bf), **kw)]


def test_bf16_calls_run_on_their_tensors_device_and_stream(lib, monkeypatch, streams):
    fake = FakeLibrary(streams)
    monkeypatch.setattr(lib, "load", lambda: fake)
    for call in bf16_calls(lib, "cuda:1"):
        call()
        assert fake.calls[-1][1:] == (1, 101), fake.calls[-1]
        call(stream=fake_stream(7, 1))
        assert fake.calls[-1][1:] == (1, 7), fake.calls[-1]
        with pytest.raises(ValueError, match="stream"):
            call(stream=fake_stream(7, 0))
    for call in bf16_calls(lib, "cuda:0")[:-1]:
        with monkeypatch.context() as m:
            taken = record_allocations(m, streams)
            call(stream=fake_stream(2))
        # the last: what the call makes (expert_ffn's arguments above come first)
        assert taken[-1] == 2, fake.calls[-1]


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
    return {b.data_ptr() for b in blocks}


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


@gpu
def test_fp8_workspace_needs_no_zeros_but_its_heads(lib):
    """Products with cut tiles and the layer, on a workspace of NaN bits behind
    its head, first for many rows and then for few."""
    g = gen(3)
    H, F, E, k = 1024, 512, 8, 2
    Wg, W1, W3, W2 = weights(g, H, F, E)
    layer = lib.MoEFp8Layer(None, Wg, W1, W3, W2, k)
    ws = lib.fp8_workspace(layer.dims(700))
    ws[lib.FP8_WORKSPACE_ZEROS:] = 0xFF
    for T in (700, 1, 130):
        x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
        _, y, q, s = lib.add_rmsnorm_fp8(x)
        got = lib.fp8_layer_forward(layer.dims(T), y, q, s, Wg, layer.routed, ws)
        clean = torch.zeros(lib.fp8_workspace_size(layer.dims(T)), dtype=torch.uint8, device="cuda")
        want = lib.fp8_layer_forward(layer.dims(T), y, q, s, Wg, layer.routed, clean)
        assert torch.equal(got, want) and bool(got.isfinite().all())
        w, w_scale = layer.routed.w2[:1], layer.routed.w2_scale[:1]
        a = q[:, :F].contiguous()
        a_scale = s[:, : F // 128].contiguous()
        assert torch.equal(lib.fp8_matmul(a, a_scale, w, w_scale, ws), lib.fp8_matmul(a, a_scale, w, w_scale, clean))
        assert lib.check(ws) == lib.MOE_OK and lib.check(clean) == lib.MOE_OK


@gpu
@pytest.mark.parametrize("bits", [8, 16])
def test_layer_graph_outlives_the_workspaces_of_eager_calls(lib, bits):
    """Captured after a warm-up, as usual; then eager calls of longer batches
    outgrow the warm-up's workspace and its memory goes elsewhere; replayed."""
    g = gen(4)
    H, F, E, k = 512, 256, 8, 2
    Wg, W1, W3, W2 = weights(g, H, F, E)
    x = torch.randn(4, H, generator=g, device="cuda").bfloat16()
    long = torch.randn(900, H, generator=g, device="cuda").bfloat16()
    layer = lib.MoEFp8Layer(None, Wg, W1, W3, W2, k) if bits == 8 else lib.MoELayer(Wg, W1, W3, W2, k)
    call = (lambda v: layer.forward(v)[0]) if bits == 8 else layer.forward
    want, want_long = call(x), call(long)
    layer._ws.clear()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = call(x)
    with torch.cuda.stream(side):
        assert torch.equal(call(long), want_long)   # before any replay
        busy = [torch.full((1 << 22,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(32)]
    torch.cuda.synchronize()
    for _ in range(2):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    assert len(busy) == 32


@gpu
@pytest.mark.parametrize("T,H,F,E,k,Fs", [(1, 512, 256, 8, 2, 0), (300, 512, 256, 8, 2, 128), (5000, 512, 128, 64, 6, 0),
                                          (700, 512, 4096, 8, 2, 0), (4500, 1024, 256, 16, 4, 0)])
def test_bf16_workspace_needs_no_zeros_but_its_error_word(lib, T, H, F, E, k, Fs):
    g = gen(5)
    Wg, W1, W3, W2 = weights(g, H, F, E)
    shared = [None] * 3 if not Fs else [t[0] for t in weights(g, H, Fs, 1)[1:]]
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    dims = lib.make_dims(T, H, F, E, k, Fs)
    clean = torch.zeros(lib.workspace_size(dims), dtype=torch.uint8, device="cuda")
    dirty = clean.clone()
    dirty[256:] = 0xFF
    want, got = (lib.layer_forward(dims, x, Wg, W1, W3, W2, ws, None, *shared) for ws in (clean, dirty))
    assert torch.equal(got, want) and lib.check(clean) == lib.MOE_OK and lib.check(dirty) == lib.MOE_OK


@gpu
def test_quantized_weights_on_a_side_stream_while_the_current_one_is_busy(lib):
    w = (torch.randn(3, 512, 256, generator=gen(6), device="cuda") * 0.02).bfloat16()
    want, want_scale = lib.fp8_quantize_weight(w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    late_fill([want.numel(), 4 * want_scale.numel()], 0xFF)
    q, scale = lib.fp8_quantize_weight(w, stream=side)
    with torch.cuda.stream(side):
        assert torch.equal(q.view(torch.uint8), want.view(torch.uint8)) and torch.equal(scale, want_scale)
    torch.cuda.synchronize()
    assert torch.equal(q.view(torch.uint8), want.view(torch.uint8)) and torch.equal(scale, want_scale)


@gpu
def test_bf16_layer_output_on_a_side_stream_while_the_current_one_is_busy(lib):
    g = gen(7)
    T, H, F, E, k = 300, 512, 256, 8, 2
    Wg, W1, W3, W2 = weights(g, H, F, E)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    layer = lib.MoELayer(Wg, W1, W3, W2, k)
    want = layer.forward(x)
    side = torch.cuda.Stream()
    layer.workspace(T, side)
    torch.cuda.synchronize()
    late_fill([want.numel() * 2] * 4, 0xFF)
    got = layer.forward(x, stream=side)
    with torch.cuda.stream(side):
        assert torch.equal(got, want)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@gpu
@pytest.mark.parametrize("call", ["norm", "matmul", "gated", "quantize_weight", "layer"])
def test_outputs_of_a_call_on_a_side_stream_are_that_streams_memory(lib, call):
    """While the current stream still has to write blocks of the outputs' sizes
    that the host has freed: outputs out of its pool would be those blocks."""
    g = gen(8)
    T, H, F, E, k = 128, 512, 256, 8, 2
    Wg, W1, W3, W2 = weights(g, H, F, E)
    layer = lib.MoEFp8Layer(None, Wg, W1, W3, W2, k)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    _, y, q, s = lib.add_rmsnorm_fp8(x)
    f, ws = layer.routed, lib.fp8_workspace(layer.dims(T))
    one = (f.w1[:1], f.w1_scale[:1])
    calls = {"norm": lambda **kw: lib.add_rmsnorm_fp8(x, residual=x, **kw),
             "matmul": lambda **kw: (lib.fp8_matmul(q, s, *one, ws, **kw),),
             "gated": lambda **kw: lib.fp8_gated(q, s, *one, *one, ws, **kw),
             "quantize_weight": lambda **kw: lib.fp8_quantize_weight(W1, **kw),
             "layer": lambda **kw: (lib.fp8_layer_forward(layer.dims(T), y, q, s, Wg, f, ws, **kw),)}
    bits = lambda ts: [t.contiguous().view(torch.uint8) for t in ts]  # noqa: E731
    want = bits(calls[call]())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = late_fill([t.numel() for t in want] * 2, 0xFF)
    got = calls[call](stream=side)
    assert not freed & {t.data_ptr() for t in got}
    with torch.cuda.stream(side):
        assert all(torch.equal(a, b) for a, b in zip(bits(got), want))
    # what the current stream's pool gives now is among them
    assert torch.empty(want[0].numel(), dtype=torch.uint8, device="cuda").data_ptr() in freed
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(bits(got), want))
