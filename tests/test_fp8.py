"""The 8-bit operators (add_rmsnorm_fp8, fp8_quantize_weight, fp8_matmul,
fp8_gated, fp8_layer_forward) against plain definitions in 64 bits.

Tolerances count roundings: half a step is eps / 2 relative (bf16 2^-8, fp16
2^-11, fp32 2^-24, e4m3 2^-4, and 2^-10 of the scale below e4m3's normal
range). A row's sum of squares is at most 90 fp32 additions deep, so the norm's
factor is within 2^-18; a product's fp32 sum of K terms is within
(K + 64) 2^-23 of the sum of the terms' magnitudes.
"""
import ctypes

import pytest
import torch

gpu = pytest.mark.gpu
BLOCK = 128
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    from token_dispatch_grouped_moe_gb300 import build, lib as L
    build.build()
    L.load()
    return L


@pytest.fixture(scope="module")
def ws(lib):
    return lib.fp8_workspace()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def spread(scale, n, dim=-1):
    return scale.double().repeat_interleave(BLOCK, dim).narrow(dim, 0, n)


def block_amax(v):
    """Largest magnitude of each row's block of 128."""
    pad = -v.shape[-1] % BLOCK
    return torch.nn.functional.pad(v, (0, pad)).unflatten(-1, (-1, BLOCK)).abs().amax(-1)


def quantized(g, R, K, spread_rows=True):
    """Random e4m3 rows with block scales of very different sizes."""
    q = (torch.randn(R, K, generator=g, device="cuda") * 100).clamp(-448, 448).to(FP8)
    s = torch.exp(torch.randn(R, -(-K // BLOCK), generator=g, device="cuda") * (1.0 if spread_rows else 0.0)) * 0.01
    return q, s


def weight(g, G, N, K):
    q = (torch.randn(G, N, K, generator=g, device="cuda") * 100).clamp(-448, 448).to(FP8)
    s = 0.0002 * torch.exp(0.5 * torch.randn(G, -(-N // BLOCK), -(-K // BLOCK), generator=g, device="cuda"))
    return q, s


def rows64(q, s):
    return q.double() * spread(s, q.shape[1])


def weight64(q, s, g):
    return q[g].double() * spread(spread(s[g], q.shape[2]), q.shape[1], 0)


def offsets_of(counts, first=0):
    o = [first]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32, device="cuda"), o


def product64(a, a_scale, w, w_scale, ends):
    """(product, sum of magnitudes) in 64 bits, NaN in rows of no group."""
    R, N = a.shape[0], w.shape[1]
    out = torch.full((R, N), float("nan"), dtype=torch.float64, device="cuda")
    mag = out.clone()
    for g in range(w.shape[0]):
        lo, hi = ends[g], ends[g + 1]
        if hi > lo:
            x, y = rows64(a[lo:hi], a_scale[lo:hi]), weight64(w, w_scale, g).T
            out[lo:hi] = x @ y
            mag[lo:hi] = x.abs() @ y.abs()
    return out, mag


# --------------------------------------------------------------- refusals --

def test_refusals_on_the_host(lib):
    """Bad arguments return a status before any CUDA call (no GPU here)."""
    L = lib.load()
    p, null, odd = ctypes.c_void_p(256), None, ctypes.c_void_p(264)
    need = lib.fp8_workspace_size()
    assert need > 0 and need % 256 == 0

    def norm(T=4, H=64, dtype=0, x=p, xs=64, res=p, rs=64, w=p, eps=1e-6, s=p, ss=64, y=p, q=p, sc=p):
        return L.moe_add_rmsnorm_fp8(T, H, dtype, x, xs, res, rs, w, eps, s, ss, y, q, sc, null)

    assert norm(T=0, x=null, q=null) == 0
    assert norm(T=-1) == 1 and norm(H=0) == 1 and norm(eps=-1.0) == 1 and norm(eps=float("nan")) == 1
    assert norm(H=40) == 2 and norm(H=32784) == 2 and norm(dtype=3) == 2 and norm(T=1 << 31) == 2
    assert norm(x=null) == 1 and norm(q=null) == 1 and norm(sc=null) == 1
    assert norm(x=odd) == 1 and norm(res=odd) == 1 and norm(w=odd) == 1 and norm(y=odd) == 1 and norm(q=odd) == 1
    assert norm(xs=63) == 1 and norm(xs=68) == 1 and norm(rs=32) == 1 and norm(ss=65) == 1

    def quant(G=2, K=64, N=64, w=p, q=p, s=p):
        return L.moe_fp8_quantize_weight(G, K, N, w, q, s, null)

    assert quant(G=0) == 1 and quant(K=0) == 1 and quant(N=-16) == 1
    assert quant(K=40) == 2 and quant(N=8) == 2 and quant(G=257) == 2
    assert quant(w=null) == 1 and quant(q=null) == 1 and quant(s=null) == 1 and quant(w=odd) == 1

    def mm(R=4, K=64, N=64, G=2, a=p, s=p, off=p, w=p, wsc=p, dt=0, out=p, ws=ctypes.c_void_p(4096), n=need):
        return L.moe_fp8_matmul(R, K, N, G, a, s, off, w, wsc, dt, out, ws, n, null)

    assert mm(R=0, a=null) == 0
    assert mm(R=-1) == 1 and mm(K=0) == 1 and mm(N=0) == 1 and mm(G=0) == 1
    assert mm(off=null) == 1                       # two groups need offsets
    assert mm(K=72) == 2 and mm(N=24) == 2 and mm(G=257) == 2 and mm(R=1 << 31) == 2 and mm(dt=1) == 2 and mm(dt=9) == 2
    assert mm(a=null) == 1 and mm(s=null) == 1 and mm(w=null) == 1 and mm(wsc=null) == 1 and mm(out=null) == 1
    assert mm(a=odd) == 1 and mm(w=odd) == 1 and mm(out=odd) == 1
    assert mm(ws=null) == 3 and mm(ws=ctypes.c_void_p(4096 + 16)) == 3 and mm(n=need - 1) == 3

    def gated(R=4, K=64, F=64, G=2, a=p, off=p, w1=p, w3=p, h=p, hs=p, ws=ctypes.c_void_p(4096), n=need):
        return L.moe_fp8_gated(R, K, F, G, a, p, off, w1, p, w3, p, h, hs, ws, n, null)

    assert gated(R=0, a=null) == 0
    assert gated(off=null) == 1 and gated(w1=null) == 1 and gated(w3=null) == 1 and gated(h=null) == 1
    assert gated(hs=null) == 1 and gated(h=odd) == 1 and gated(F=8) == 2 and gated(n=need - 1) == 3


def test_layer_refusals_on_the_host(lib):
    L = lib.load()
    p, null = ctypes.c_void_p(256), None
    d = lib.make_dims(8, 64, 64, 8, 2)
    need = lib.fp8_workspace_size(d)
    assert need > lib.fp8_workspace_size() + lib.workspace_size(d) - 256
    assert lib.fp8_workspace_size(lib.make_dims(8, 60, 64, 8, 2)) == 0
    full = lib.Fp8Ffn(*([256] * 6))
    part = lib.Fp8Ffn(*([256] * 5), None)

    def layer(dims=d, x=p, xq=p, xs=p, Wg=p, f=full, fs=None, out=p, ws=ctypes.c_void_p(4096), n=need):
        return L.moe_fp8_layer_forward(ctypes.byref(dims), x, xq, xs, Wg, null, None,
                                       None if f is None else ctypes.byref(f),
                                       None if fs is None else ctypes.byref(fs), out, None, ws, n, null)

    assert L.moe_fp8_layer_forward(None, p, p, p, p, null, None, None, None, p, None, p, need, null) == 1
    assert layer(x=null) == 1 and layer(xq=null) == 1 and layer(xs=null) == 1 and layer(Wg=null) == 1
    assert layer(f=None) == 1 and layer(f=part) == 1 and layer(out=null) == 1
    assert layer(ws=null) == 3 and layer(n=need - 1) == 3
    shared = lib.make_dims(8, 64, 64, 8, 2, 64)
    assert layer(dims=shared, n=lib.fp8_workspace_size(shared)) == 1      # the shared expert's weights
    empty = lib.make_dims(0, 64, 64, 8, 2)
    assert layer(dims=empty, x=null, n=lib.fp8_workspace_size(empty)) == 0


def test_binding_checks_tensors(lib):
    """Wrong shapes, types and layouts are refused by the binding (on CPU
    tensors: nothing reaches the library)."""
    a = torch.zeros(4, 64, dtype=torch.float32).to(FP8)
    s = torch.zeros(4, 1)
    w, wsc = torch.zeros(2, 32, 64).to(FP8), torch.zeros(2, 1, 1)
    off = torch.zeros(3, dtype=torch.int32)
    ws = torch.zeros(16, dtype=torch.uint8)
    bad = [
        lambda: lib.fp8_matmul(a.float(), s, w, wsc, ws, offsets=off),
        lambda: lib.fp8_matmul(a, s[:3], w, wsc, ws, offsets=off),
        lambda: lib.fp8_matmul(a, s, w[:, :, :32], wsc, ws, offsets=off),
        lambda: lib.fp8_matmul(a, s, w, wsc[:1], ws, offsets=off),
        lambda: lib.fp8_matmul(a, s, w, wsc, ws, offsets=off[:2]),
        lambda: lib.fp8_matmul(a, s, w, wsc, ws, offsets=off.long()),
        lambda: lib.fp8_matmul(a, s, w, wsc, ws, offsets=off, out_dtype=torch.float16),
        lambda: lib.fp8_matmul(a, s, w, wsc, ws, offsets=off, out=torch.zeros(4, 33)),
        lambda: lib.fp8_gated(a, s, w, wsc, w[:, :16], wsc, ws, offsets=off),
        lambda: lib.add_rmsnorm_fp8(torch.zeros(4, 64, dtype=torch.int32)),
        lambda: lib.add_rmsnorm_fp8(torch.zeros(4, 64), weight=torch.zeros(32)),
        lambda: lib.add_rmsnorm_fp8(torch.zeros(4, 64), residual=torch.zeros(4, 64, dtype=torch.float16)),
        lambda: lib.add_rmsnorm_fp8(torch.zeros(64, 4).t()),
        lambda: lib.fp8_quantize_weight(torch.zeros(2, 64, 64)),
    ]
    bad += [
        lambda: lib.fp8_matmul(a[0], s, w, wsc, ws, offsets=off),
        lambda: lib.fp8_matmul(a, s, w[0], wsc, ws, offsets=off),
        lambda: lib.fp8_matmul(a, None, w, wsc, ws, offsets=off),
        lambda: lib.fp8_matmul(a, s, w, wsc, ws.int(), offsets=off),
        lambda: lib.fp8_matmul(a, s, w, wsc, ws, offsets=off),           # right, but not on a GPU
        lambda: lib.fp8_gated(a, s, w, wsc, w, wsc[:, :0], ws, offsets=off),
        lambda: lib.add_rmsnorm_fp8(torch.zeros(64)),
        lambda: lib.add_rmsnorm_fp8([1.0]),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(lib.MoeError):
        lib.fp8_workspace(lib.make_dims(8, 60, 64, 8, 2))


# ------------------------------------------------------------------- norm --

def check_quantized(q, scale, ref, err):
    """q, scale against the 64-bit values ref, known within err."""
    amax = block_amax(ref).clamp(min=2.0 ** -100)
    amax_err = block_amax(err)
    assert bool(((scale.double() - amax / 448).abs() <= amax_err / 448 + amax / 448 * 2 ** -22).all())
    s = spread(scale, ref.shape[1])
    got = q.double() * s
    bound = (ref.abs() + err) * (2 ** -4 + 2 ** -20) + s * 2 ** -10 + err
    assert bool(((got - ref).abs() <= bound).all())


def norm64(x, res, w, eps):
    r = x.double() + (res.double() if res is not None else 0)
    y = r / torch.sqrt(r.square().mean(-1, keepdim=True) + eps)
    return r, y * w.double() if w is not None else y


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,H", [(1, 16), (3, 64), (5, 128), (2, 144), (7, 2048), (33, 3584), (4, 4096), (3, 4112),
                                 (2, 8208), (2, 16400), (3, 32768), (1, 4096)])
@pytest.mark.parametrize("parts", ["x", "x+res", "x+res*w"])
def test_norm(lib, dtype, T, H, parts):
    g = gen(T * H)
    x = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    res = (4 * torch.randn(T, H, generator=g, device="cuda")).to(dtype) if "res" in parts else None
    w = (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(dtype) if "w" in parts else None
    s, y, q, scale = lib.add_rmsnorm_fp8(x, w, residual=res, eps=1e-6)
    r64, y64 = norm64(x, res, w, 1e-6)
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).tiny * torch.finfo(dtype).eps
    if res is None:
        assert s is None
    else:
        assert s.dtype == dtype and bool(((s.double() - r64).abs() <= r64.abs() * (half + 2 ** -23) + tiny).all())
    assert bool(((y.double() - y64).abs() <= y64.abs() * (half + 2 ** -18) + tiny).all())
    check_quantized(q, scale, y64, y64.abs() * 2 ** -18)
    assert lib.add_rmsnorm_fp8(x, w, residual=res, eps=1e-6, want_y=False)[1] is None


@gpu
def test_norm_strided_rows_and_in_place(lib):
    g = gen(5)
    wide = torch.randn(9, 640, generator=g, device="cuda").bfloat16()
    x, res = wide[:, :256], wide[:, 320:576]
    want = lib.add_rmsnorm_fp8(x.contiguous(), residual=res.contiguous())
    keep = wide.clone()
    got = lib.add_rmsnorm_fp8(x, residual=res, sum_out=res)
    for a, b in zip(want, got):
        assert torch.equal(a.view(torch.uint8) if a.dtype == FP8 else a, b.view(torch.uint8) if b.dtype == FP8 else b)
    assert torch.equal(wide[:, 320:576], want[0])
    assert torch.equal(wide[:, :320], keep[:, :320]) and torch.equal(wide[:, 576:], keep[:, 576:])
    wide.copy_(keep)
    got = lib.add_rmsnorm_fp8(x, residual=res, sum_out=x)
    assert torch.equal(got[0], want[0]) and torch.equal(wide[:, :256], want[0])
    with pytest.raises(lib.MoeError):
        lib.add_rmsnorm_fp8(wide[:, 4:260])   # rows start 8 bytes off a 16-byte boundary


@gpu
def test_norm_special_rows(lib):
    """Rows of zeros, of the type's extremes, with NaN or infinity; no rows."""
    H = 384
    x = torch.zeros(6, H, device="cuda")
    x[1] = 1e-30
    x[2, 5] = float("nan")
    x[3, 200] = float("inf")
    x[4] = torch.randn(H, generator=gen(1), device="cuda") * 1e15
    x[5, 130] = 3.0   # two blocks of zeros around one value
    _, y, q, scale = lib.add_rmsnorm_fp8(x, eps=1e-6)
    assert bool((y[0] == 0).all()) and bool((q[0].float() == 0).all()) and bool((scale[0] == 2.0 ** -100 / 448).all())
    ref = norm64(x[[1, 4, 5]], None, None, 1e-6)[1]
    assert bool(((y[[1, 4, 5]].double() - ref).abs() <= ref.abs() * 2 ** -17).all())
    check_quantized(q[[1, 4, 5]], scale[[1, 4, 5]], ref, ref.abs() * 2 ** -18)
    # a NaN spoils its row's mean, so the whole row; an infinity leaves 0 beside itself
    assert bool(y[2].isnan().all()) and bool(scale[2].isnan().all()) and bool(q[2].float().isnan().all())
    assert bool(y[3, 200].isnan()) and bool(scale[3, 1].isnan()) and bool(q[3, 128:256].float().isnan().all())
    assert bool((q[3, :128].float() == 0).all()) and bool((q[3, 256:].float() == 0).all())
    s, y, q, scale = lib.add_rmsnorm_fp8(x[:0], residual=x[:0])
    assert q.shape == (0, H) and scale.shape == (0, 3)


@gpu
def test_norm_long_batch(lib):
    """More elements than 32 bits count."""
    T, H = 70000, 32768
    x = torch.ones(1, H, dtype=torch.bfloat16, device="cuda").expand(T, H).contiguous()
    x[-1, ::2] = 3
    _, _, q, scale = lib.add_rmsnorm_fp8(x, want_y=False)
    ref = norm64(x[-1:], None, None, 1e-6)[1]
    check_quantized(q[-1:], scale[-1:], ref, ref.abs() * 2 ** -18)
    assert torch.equal(q[0].view(torch.uint8), q[T // 2].view(torch.uint8))
    assert float(q[T - 2].float().min()) == 448.0 and bool((scale[: T - 1] == scale[0]).all())


# ---------------------------------------------------------------- weights --

@gpu
@pytest.mark.parametrize("G,K,N", [(1, 16, 16), (3, 128, 128), (2, 144, 272), (4, 1408, 512), (2, 512, 1408),
                                   (1, 2048, 48), (2, 64, 16)])
def test_quantize_weight(lib, G, K, N):
    w = (torch.randn(G, K, N, generator=gen(K + N), device="cuda") * 0.02).bfloat16()
    w[0, :16, :16] = 0
    q, scale = lib.fp8_quantize_weight(w)
    t = w.double().transpose(1, 2)
    pad = torch.nn.functional.pad(t, (0, -K % BLOCK, 0, -N % BLOCK))
    amax = pad.unflatten(2, (-1, BLOCK)).unflatten(1, (-1, BLOCK)).abs().amax((2, 4)).clamp(min=2.0 ** -100)
    assert q.shape == (G, N, K) and scale.shape == amax.shape
    assert torch.equal(scale, (amax / 448).float())   # the quotient, rounded once
    s = spread(spread(scale, K), N, 1)
    err = (q.double() * s - t).abs()
    assert bool((err <= t.abs() * (2 ** -4 + 2 ** -20) + s * 2 ** -10).all())


# --------------------------------------------------------------- products --

PRODUCTS = [   # K, N, rows of each group
    (16, 16, [1]), (128, 16, [0, 1, 0]), (48, 64, [5]), (128, 128, [128]), (144, 144, [3, 0, 130]),
    (256, 256, [129, 1]), (2048, 272, [0, 0, 7]), (1408, 2048, [1] * 6 + [0] * 10), (400, 400, [127, 128, 129, 0, 300]),
    (4096, 1024, [1]), (4096, 1024, [40]), (14336, 256, [1, 0, 1]), (14336, 256, [2, 128, 1]), (20480, 384, [333]),
    (2048, 1408, [90 + (7 * i) % 13 for i in range(64)]), (512, 128, [1] * 256), (256, 512, [3] * 255 + [1000]),
    (256, 320, [2085]), (400, 272, [3000, 0, 5001, 100]), (4096, 14336, [1, 1]), (2048, 40960, [17]), (16384, 512, [1]),
    (8192, 272, [130]), (8192, 144, [20, 40, 0, 33]), (1024, 2064, [1]), (1040, 2064, [1]),
]


def check_product(out, ref, mag, K, dtype):
    half = torch.finfo(dtype).eps / 2
    rows = ~ref[:, 0].isnan()
    out, ref, mag = out[rows].double(), ref[rows], mag[rows]
    assert bool(((out - ref).abs() <= ref.abs() * half + mag * ((K + 64) * 2.0 ** -23)).all())
    # and over all values: K roundings that do not conspire add up as their root
    rel = float((out - ref).norm() / ref.norm())
    assert rel <= half + 4 * K ** 0.5 * 2 ** -24, rel


@gpu
@pytest.mark.parametrize("K,N,counts", PRODUCTS, ids=lambda v: str(v) if isinstance(v, int) else f"{len(v)}g{sum(v)}r")
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_matmul(lib, ws, K, N, counts, dtype):
    g = gen(K * N + sum(counts))
    R = sum(counts)
    a, a_scale = quantized(g, R, K)
    w, w_scale = weight(g, len(counts), N, K)
    off, ends = offsets_of(counts)
    out = torch.full((R, N), float("nan"), dtype=dtype, device="cuda")
    lib.fp8_matmul(a, a_scale, w, w_scale, ws, offsets=off, out_dtype=dtype, out=out)
    assert lib.check(ws) == lib.MOE_OK
    check_product(out, *product64(a, a_scale, w, w_scale, ends), K, dtype)
    again = lib.fp8_matmul(a, a_scale, w, w_scale, ws, offsets=off, out_dtype=dtype)
    assert torch.equal(out, again)
    if len(counts) == 1:
        dense = lib.fp8_matmul(a, a_scale, w, w_scale, ws, out_dtype=dtype)
        assert torch.equal(out, dense)


@gpu
def test_matmul_rows_outside_groups_and_bad_offsets(lib, ws):
    g = gen(3)
    K, N, R = 256, 320, 50
    a, a_scale = quantized(g, R, K)
    w, w_scale = weight(g, 3, N, K)
    off, ends = offsets_of([10, 0, 20], first=5)
    out = torch.full((R, N), -7.0, dtype=torch.float32, device="cuda")
    lib.fp8_matmul(a, a_scale, w, w_scale, ws, offsets=off, out_dtype=torch.float32, out=out)
    assert lib.check(ws) == lib.MOE_OK
    assert bool((out[:5] == -7).all()) and bool((out[35:] == -7).all())
    check_product(out, *product64(a, a_scale, w, w_scale, ends), K, torch.float32)
    # no rows at all, then offsets that decrease, leave the rows, or start below them
    for bad, status in ([0, 0, 0, 0], 0), ([0, 30, 20, 50], 6), ([0, 10, 20, 51], 6), ([-1, 10, 20, 30], 6):
        out.fill_(-7.0)
        o = torch.tensor(bad, dtype=torch.int32, device="cuda")
        lib.fp8_matmul(a, a_scale, w, w_scale, ws, offsets=o, out_dtype=torch.float32, out=out)
        assert lib.check(ws) == status
        assert bool((out == -7).all())
        h, hs = lib.fp8_gated(a, a_scale, w, w_scale, w, w_scale, ws, offsets=o)
        assert lib.check(ws) == status
    assert lib.fp8_matmul(a[:0], a_scale[:0], w, w_scale, ws, offsets=off).shape == (0, N)


@gpu
def test_matmul_nan_stays_in_its_row(lib, ws):
    g = gen(4)
    a, a_scale = quantized(g, 20, 512)
    w, w_scale = weight(g, 1, 256, 512)
    want = lib.fp8_matmul(a, a_scale, w, w_scale, ws, out_dtype=torch.float32)
    a_scale[3, 1] = float("nan")
    a[7, 100] = float("nan")
    a_scale[9] = float("inf")
    got = lib.fp8_matmul(a, a_scale, w, w_scale, ws, out_dtype=torch.float32)
    assert bool(got[3].isnan().all()) and bool(got[7].isnan().all()) and not bool(got[9].isfinite().any())
    rows = [i for i in range(20) if i not in (3, 7, 9)]
    assert torch.equal(got[rows], want[rows])


@gpu
def test_matmul_long_output(lib, ws):
    """An output of more elements than 32 bits count."""
    g = gen(6)
    R, K, N = 140001, 128, 16384
    a, a_scale = quantized(g, R, K)
    w, w_scale = weight(g, 2, N, K)
    off = torch.tensor([0, 139000, R], dtype=torch.int32, device="cuda")
    out = lib.fp8_matmul(a, a_scale, w, w_scale, ws, offsets=off)
    assert lib.check(ws) == lib.MOE_OK
    for lo, e in ((138990, 0), (R - 10, 1)):
        x, y = rows64(a[lo: lo + 10], a_scale[lo: lo + 10]), weight64(w, w_scale, e).T
        check_product(out[lo: lo + 10], x @ y, x.abs() @ y.abs(), K, torch.bfloat16)


@gpu
@pytest.mark.parametrize("K,F,counts", [(16, 16, [1]), (128, 64, [0, 3]), (144, 144, [3, 0, 130]), (256, 192, [129, 1]),
                                        (512, 128, [128]), (2048, 1408, [1] * 6 + [0] * 10), (4096, 272, [1, 1]),
                                        (4096, 1024, [40]), (8192, 128, [2, 128, 1]), (400, 400, [127, 128, 129, 0, 300]),
                                        (2048, 1408, [90 + (7 * i) % 13 for i in range(64)]), (128, 256, [1] * 256),
                                        (256, 272, [600]), (400, 144, [1000, 0, 257, 900]), (4096, 14336, [1, 0, 2])],
                         ids=lambda v: str(v) if isinstance(v, int) else f"{len(v)}g{sum(v)}r")
def test_gated(lib, ws, K, F, counts):
    g = gen(K + F + sum(counts))
    R = sum(counts)
    a, a_scale = quantized(g, R, K, spread_rows=False)
    w1, s1 = weight(g, len(counts), F, K)
    w3, s3 = weight(g, len(counts), F, K)
    off, ends = offsets_of(counts)
    h, scale = lib.fp8_gated(a, a_scale, w1, s1, w3, s3, ws, offsets=off)
    assert lib.check(ws) == lib.MOE_OK
    p1, m1 = product64(a, a_scale, w1, s1, ends)
    p3, m3 = product64(a, a_scale, w3, s3, ends)
    act = p1 * torch.sigmoid(p1)
    ref = act * p3
    step = (K + 64) * 2.0 ** -23
    # |silu'| <= 1.1; the activation's own roundings grow with |p1| (its exponent's argument)
    err = 1.1 * m1 * step * p3.abs() + act.abs() * m3 * step + ref.abs() * (2 ** -20 + p1.abs() * 2 ** -21)
    check_quantized(h, scale, ref, err)
    again = lib.fp8_gated(a, a_scale, w1, s1, w3, s3, ws, offsets=off)
    assert torch.equal(h.view(torch.uint8), again[0].view(torch.uint8)) and torch.equal(scale, again[1])


@gpu
def test_gated_large_arguments(lib, ws):
    """Activations far to either side: silu is -0 or the argument itself."""
    K, F = 128, 128
    a = torch.ones(2, K, device="cuda").to(FP8)
    a[1] = (-torch.ones(K, device="cuda")).to(FP8)
    a_scale = torch.full((2, 1), 100.0, device="cuda")
    w = torch.ones(1, F, K, device="cuda").to(FP8)
    w_scale = torch.ones(1, 1, 1, device="cuda")
    h, scale = lib.fp8_gated(a, a_scale, w, w_scale, w, w_scale, ws)
    assert bool((h[0].float() == 448).all()) and abs(float(scale[0, 0]) / (12800.0 ** 2 / 448) - 1) <= 2 ** -20
    assert bool((h[1].float() == 0).all()) and float(scale[1, 0]) == float(torch.tensor(2.0 ** -100 / 448))


@gpu
def test_streams_and_graph(lib):
    """Calls on another stream than the default, and captured into a graph and
    replayed on new inputs."""
    g = gen(8)
    K, F, R = 1024, 256, 6
    own = lib.fp8_workspace()
    a, a_scale = quantized(g, R, K)
    b, b_scale = quantized(g, R, K)
    w1, s1 = weight(g, 1, F, K)
    w3, s3 = weight(g, 1, F, K)
    x = torch.randn(R, K, generator=g, device="cuda").bfloat16()

    def both(p, p_scale, **kw):
        h, hs = lib.fp8_gated(p, p_scale, w1, s1, w3, s3, own, **kw)
        return [t.view(torch.uint8) if t.dtype == FP8 else t
                for t in (h, hs, lib.fp8_matmul(p, p_scale, w1, s1, own, **kw), *lib.add_rmsnorm_fp8(x, **kw)[1:])]

    want, want_b = both(a, a_scale), both(b, b_scale)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = both(a, a_scale)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    # a stream given by argument: the outputs' memory is that stream's, so memory
    # that the current stream frees and takes again cannot be the same
    torch.cuda._sleep(1000000)
    got = both(a, a_scale, stream=side)
    busy = [torch.full_like(t, 3) for t in got]
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got)) and len(busy) == len(got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = both(a, a_scale)
    a.copy_(b)
    a_scale.copy_(b_scale)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want_b, got))
    assert lib.check(own) == lib.MOE_OK


# ------------------------------------------------------------------ layer --

@gpu
@pytest.mark.parametrize("T,H,F,E,k,Fs", [(1, 512, 256, 8, 2, 0), (37, 512, 192, 8, 2, 0), (300, 256, 320, 64, 6, 128),
                                          (700, 2048, 128, 16, 4, 256)])
def test_layer(lib, T, H, F, E, k, Fs):
    """The layer equals its parts bit for bit (router, sort, gated product,
    product, rank-order sum) and the 64-bit layer on the same 8-bit weights."""
    g = gen(T + H)
    rnd = lambda *s, sigma=0.02: (torch.randn(*s, generator=g, device="cuda") * sigma).bfloat16()  # noqa: E731
    Wg, W1, W3, W2 = rnd(H, E), rnd(E, H, F, sigma=0.05), rnd(E, H, F, sigma=0.05), rnd(E, F, H, sigma=0.05)
    shared = (rnd(H, Fs, sigma=0.05), rnd(H, Fs, sigma=0.05), rnd(Fs, H, sigma=0.05)) if Fs else (None, None, None)
    nw = (1 + rnd(H, sigma=0.2)).bfloat16()
    layer = lib.MoEFp8Layer(nw, Wg, W1, W3, W2, k, None, *shared)
    x, res = rnd(T, H, sigma=1.0), rnd(T, H, sigma=2.0)
    dims = layer.dims(T)
    rt = lib.routing_buffers(dims, x.device)
    out, stream = layer.forward(x, res, routing=rt)
    ws = layer.workspace(T)
    assert lib.check(ws) == lib.MOE_OK
    out2, _ = layer.forward(x, res)
    assert torch.equal(out, out2)

    r, y, q, qs = lib.add_rmsnorm_fp8(x, nw, residual=res)
    assert torch.equal(stream, r)
    idx, tw = lib.route(dims, y, Wg)
    assert torch.equal(idx, rt.topk_idx)
    src = rt.src_row.long()
    token = src // k
    own = lib.fp8_workspace()
    f = layer.routed
    h, hs = lib.fp8_gated(q.view(torch.uint8)[token].view(FP8), qs[token], f.w1, f.w1_scale, f.w3, f.w3_scale, own,
                          offsets=rt.offsets)
    p = lib.fp8_matmul(h, hs, f.w2, f.w2_scale, own, offsets=rt.offsets, out_dtype=torch.float32)
    p = rt.topk_w.view(-1)[src][:, None] * p
    slots = torch.empty_like(p)
    slots[src] = p                                  # by assignment t k + j
    slots = list(slots.view(T, k, H).unbind(1))
    if Fs:
        s = layer.shared
        h, hs = lib.fp8_gated(q, qs, s.w1, s.w1_scale, s.w3, s.w3_scale, own)
        slots.append(lib.fp8_matmul(h, hs, s.w2, s.w2_scale, own, out_dtype=torch.float32))
    total = slots[0]
    for v in slots[1:]:
        total = total + v
    assert torch.equal(out, total.bfloat16())

    # 64 bits, on the same quantized operands; h rounded to e4m3 where it is exact
    def ffn64(xr, f, e):
        h = xr @ weight64(f.w1, f.w1_scale, e).T
        h = h * torch.sigmoid(h) * (xr @ weight64(f.w3, f.w3_scale, e).T)
        s = spread(block_amax(h) / 448, h.shape[1])
        _, ex = torch.frexp(h / s)
        step = torch.exp2((ex - 1).clamp(min=-6).double() - 3)
        return (torch.round(h / s / step) * step * s) @ weight64(f.w2, f.w2_scale, e).T

    xr = rows64(q, qs)
    ref = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = (rt.topk_idx == e).nonzero(as_tuple=True)
        if len(t):
            ref.index_add_(0, t, rt.topk_w[t, j].double()[:, None] * ffn64(xr[t], f, e))
    if Fs:
        ref += ffn64(xr, layer.shared, 0)
    # a value of h at a rounding border may go the other way: 2^-8 beside the output's 2^-8
    assert float((out.double() - ref).norm() / ref.norm()) <= 2 ** -7


@gpu
def test_layer_gating_variants(lib):
    """No renormalisation, and a sigmoid-gated shared expert, as moe_layer_forward_ex has them."""
    T, H, F, E, k, Fs = 65, 256, 128, 8, 2, 128
    g = gen(11)
    rnd = lambda *s, sigma=0.05: (torch.randn(*s, generator=g, device="cuda") * sigma).bfloat16()  # noqa: E731
    Wg, W1, W3, W2 = rnd(H, E), rnd(E, H, F), rnd(E, H, F), rnd(E, F, H)
    W1s, W3s, W2s, wsg = rnd(H, Fs), rnd(H, Fs), rnd(Fs, H), rnd(H)
    layer = lib.MoEFp8Layer(None, Wg, W1, W3, W2, k, None, W1s, W3s, W2s)
    x = rnd(T, H, sigma=1.0)
    _, y, q, qs = lib.add_rmsnorm_fp8(x)
    dims, ws = layer.dims(T), layer.workspace(T)

    def run(**kw):
        out = lib.fp8_layer_forward(dims, y, q, qs, Wg, layer.routed, ws, shared=layer.shared, **kw)
        assert lib.check(ws) == lib.MOE_OK
        return out.double()

    def bf16(**kw):
        w = lib.workspace(dims)
        return lib.layer_forward(dims, y, Wg, W1, W3, W2, w, W1s=W1s, W3s=W3s, W2s=W2s, **kw).double()

    for kw in ({}, {"renormalize": False}, {"shared_gate": wsg}, {"renormalize": False, "shared_gate": wsg}):
        a, b = run(**kw), bf16(**kw)
        # e4m3 activations, weights and h: three roundings of at most 2^-4, as independent errors
        assert float((a - b).norm() / b.norm()) <= 2 ** -4 * 3 ** 0.5
    assert float((run(renormalize=False) - run()).norm()) > 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lib.fp8_layer_forward(dims, y, q, qs, Wg, layer.routed, ws, shared=layer.shared, stream=side)
    side.synchronize()
    assert torch.equal(got.double(), run())
    with pytest.raises(ValueError):
        run(shared_gate=wsg[:64])
