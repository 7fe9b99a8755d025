"""The layer on 8-bit experts where its second product, weighted and scattered to
slots, runs as CTA pairs, in tiles of 128 columns, or cut along K; with the
tensor-core router in front; and its workspace.

The layer is held to its parts bit for bit: the parts take the same kernels on
the same rows (tests of each against 64 bits: test_fp8.py, test_fp8_forms.py), and
weighting, scattering and the sum in rank order are fp32 operations with one
result.
"""
import pytest
import torch

from test_fp8 import gen

gpu = pytest.mark.gpu
FP8 = torch.float8_e4m3fn
WIDE, NARROW, PAIR = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from token_dispatch_grouped_moe_gb300 import build, lib as L
    build.build()
    L.load()
    return L


@pytest.mark.parametrize("T,H,F,E,k,Fs", [(1, 64, 64, 8, 2, 0), (8, 64, 64, 8, 2, 64), (129, 512, 192, 8, 2, 128),
                                          (32768, 2048, 1408, 64, 6, 2816), (8192, 4096, 14336, 8, 2, 0)])
def test_workspace_is_the_products_and_the_bf16_layers(lib, T, H, F, E, k, Fs):
    """The quantized rows and h take the memory that the bf16 layer has for its
    own: nothing beside the two workspaces."""
    dims = lib.make_dims(T, H, F, E, k, Fs)
    assert lib.fp8_workspace_size(dims) <= lib.fp8_workspace_size() + lib.workspace_size(dims) + 255
    # where the rows' scales lie, behind the rows: in the other half of their buffer
    for rows, n in (T * k, H), (T * k, F), (T, Fs):
        assert rows * n + rows * -(-n // 128) * 4 <= rows * n * 2


def make_layer(lib, g, H, F, E, k, Fs):
    rnd = lambda *s, sigma=0.05: (torch.randn(*s, generator=g, device="cuda") * sigma).bfloat16()  # noqa: E731
    shared = (rnd(H, Fs), rnd(H, Fs), rnd(Fs, H)) if Fs else (None, None, None)
    return lib.MoEFp8Layer(None, rnd(H, E, sigma=0.02), rnd(E, H, F), rnd(E, H, F), rnd(E, F, H), k, None, *shared)


def parts_of(lib, layer, y, q, qs, rt, out=torch.float32):
    """The routed slots [k][T, H] and the shared expert's rows [T, H] (or None)."""
    T, H = y.shape
    k, f, own = layer.k, layer.routed, lib.fp8_workspace()
    src = rt.src_row.long()
    token = src // k
    h, hs = lib.fp8_gated(q.view(torch.uint8)[token].view(FP8), qs[token], f.w1, f.w1_scale, f.w3, f.w3_scale, own,
                          offsets=rt.offsets)
    p = lib.fp8_matmul(h, hs, f.w2, f.w2_scale, own, offsets=rt.offsets, out_dtype=out)
    slots = torch.empty_like(p)
    slots[src] = rt.topk_w.view(-1)[src][:, None] * p
    slots = list(slots.view(T, k, H).unbind(1))
    if layer.shared is None:
        return slots, None
    s = layer.shared
    h, hs = lib.fp8_gated(q, qs, s.w1, s.w1_scale, s.w3, s.w3_scale, own)
    return slots, lib.fp8_matmul(h, hs, s.w2, s.w2_scale, own, out_dtype=out)


def total(slots):
    r = slots[0]
    for v in slots[1:]:
        r = r + v
    return r


# T, H, F, E, k, F_shared; the forms of the routed gated product and the second product
LAYERS = [
    (8300, 2048, 256, 8, 2, 0, PAIR, PAIR),          # 2075 rows an expert
    (8300, 2048, 192, 8, 2, 256, PAIR, PAIR),        # and a shared expert of 8300 rows
    (4500, 512, 128, 64, 6, 0, WIDE, WIDE),          # the tensor-core router, 422 rows an expert
    (9000, 1024, 128, 16, 4, 128, PAIR, PAIR),
    (1, 1024, 14336, 8, 2, 0, WIDE, WIDE),           # one token on wide experts: K = 14336 cut
    (5, 512, 14336, 8, 2, 8192, WIDE, WIDE),
    (64, 1024, 8192, 4, 2, 0, WIDE, NARROW),         # tiles of 128 columns, cut
    (700, 256, 1024, 4, 1, 0, WIDE, NARROW),
]


def test_forms_of_the_layers_below(lib):
    for T, H, F, E, k, Fs, gated, product in LAYERS:
        assert lib.fp8_form_selftest(T * k, H, F, E, True) == gated, (T, H, F)
        assert lib.fp8_form_selftest(T * k, F, H, E) == product, (T, H, F)
    # the tensor-core router from 4096 tokens on
    assert lib.layer_plan(lib.make_dims(4500, 512, 128, 64, 6)).router == lib.ROUTER_TENSOR


@gpu
@pytest.mark.parametrize("T,H,F,E,k,Fs", [c[:6] for c in LAYERS])
def test_layer_equals_its_parts(lib, T, H, F, E, k, Fs):
    g = gen(T + H + F)
    layer = make_layer(lib, g, H, F, E, k, Fs)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    rt = lib.routing_buffers(layer.dims(T), x.device)
    out, _ = layer.forward(x, routing=rt)
    assert lib.check(layer.workspace(T)) == lib.MOE_OK
    _, y, q, qs = lib.add_rmsnorm_fp8(x)
    assert torch.equal(rt.topk_idx, lib.route(layer.dims(T), y, layer.Wg)[0])
    slots, shared = parts_of(lib, layer, y, q, qs, rt)
    assert torch.equal(out, total(slots + ([shared] if shared is not None else [])).bfloat16())
    assert torch.equal(out, layer.forward(x)[0])


@gpu
@pytest.mark.parametrize("T,H,F,E,k,Fs", [(2304, 2048, 128, 8, 2, 256), (3, 512, 128, 8, 2, 14336), (100, 256, 128, 8, 2, 512)])
def test_layer_with_a_gated_shared_expert(lib, T, H, F, E, k, Fs):
    """The shared expert's rows weighted in token order: by pairs, cut along K,
    and in tiles of 128 columns."""
    assert lib.fp8_form_selftest(T, Fs, H) == {2304: PAIR, 3: WIDE, 100: NARROW}[T]
    g = gen(T + Fs)
    layer = make_layer(lib, g, H, F, E, k, Fs)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    wsg = (torch.randn(H, generator=g, device="cuda") * 0.05).bfloat16()
    _, y, q, qs = lib.add_rmsnorm_fp8(x)
    dims, ws = layer.dims(T), layer.workspace(T)
    rt = lib.routing_buffers(dims, x.device)
    out = lib.fp8_layer_forward(dims, y, q, qs, layer.Wg, layer.routed, ws, shared=layer.shared, routing=rt,
                                shared_gate=wsg)
    assert lib.check(ws) == lib.MOE_OK
    slots, shared = parts_of(lib, layer, y, q, qs, rt)
    routed = total(slots).double()
    dot = (y.double() * wsg.double()).sum(1)
    gate = torch.sigmoid(dot)[:, None]
    ref = routed + gate * shared.double()
    # the gate: a fp32 sum of H terms (sigmoid' <= 1/4) and a few roundings of its own; a
    # product, a sum and the output's rounding
    gate_err = ((y.double() * wsg.double()).abs().sum(1) * (H + 8) * 2.0 ** -26 + 2.0 ** -20)[:, None]
    err = gate_err * shared.double().abs() + (routed.abs() + (gate * shared).abs()) * 2.0 ** -22
    assert bool(((out.double() - ref).abs() <= (ref.abs() + err) * 2.0 ** -8 + err).all())
