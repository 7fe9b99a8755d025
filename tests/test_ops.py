"""route_logits, linear and combine_rows against plain definitions in 64 bits.

Tolerances count roundings: half a step is eps / 2 relative (bf16 2^-8, fp16
2^-11, fp32 2^-24). A softmax score is within (|l - max| / 2 + 20) 2^-23 of itself (the
exponent's rounding, e^x, the sum of 256), a sigmoid score within 10 * 2^-23, a
renormalized weight within twice that and the rounding of a sum of 8; the tests keep
|l - max| below 24: 72 * 2^-23 bounds them all. A product's fp32 sum of K terms is
within (K + 64) 2^-23 of the sum of the terms' magnitudes; activations are at most
1.13 times as steep as their argument, and their own error is below 2^-20 of it.
"""
import ctypes
import math

import pytest
import torch

gpu = pytest.mark.gpu
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
WEIGHT_TOL = 72 * 2.0 ** -23


@pytest.fixture(scope="module")
def lib():
    from token_dispatch_grouped_moe_gb300 import build, lib as L
    build.build()
    L.load()
    return L


@pytest.fixture(scope="module")
def ws(lib):
    return lib.linear_workspace()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


# --------------------------------------------------------------- refusals --

def test_route_refusals_on_the_host(lib):
    """Bad arguments return a status before any CUDA call (no GPU here)."""
    L = lib.load()
    p, null, odd = ctypes.c_void_p(256), None, ctypes.c_void_p(258)

    def call(T=4, E=64, k=6, dtype=2, logits=p, stride=64, idx=p, w=p, scoring=True, scores=1, bias=256, groups=8,
             top_groups=4, group_top=2, renorm=1, scale=1.0):
        c = lib.Scoring(scores, bias, groups, top_groups, group_top, renorm, scale)
        return L.moe_route_logits(T, E, k, dtype, logits, stride, ctypes.byref(c) if scoring else None, idx, w, null)

    assert call(T=0, logits=null, idx=null, w=null) == 0
    assert call(T=-1) == 1 and call(E=0) == 1 and call(k=0) == 1 and call(k=65) == 1 and call(scores=2) == 1
    assert call(groups=0) == 1 and call(groups=7) == 1 and call(top_groups=0) == 1 and call(top_groups=9) == 1
    assert call(group_top=0) == 1 and call(group_top=3) == 1 and call(E=8, k=1, group_top=2) == 1
    assert call(E=8, k=3, groups=4, top_groups=1) == 1             # two experts to choose from
    assert call(scale=float("nan")) == 1 and call(scale=float("inf")) == 1
    assert call(k=9) == 2 and call(E=264, stride=264) == 2 and call(dtype=3) == 2 and call(T=1 << 31) == 2
    assert call(E=128, stride=128, groups=64, top_groups=64) == 2
    assert call(logits=null) == 1 and call(idx=null) == 1 and call(w=null) == 1 and call(stride=63) == 1
    assert call(logits=odd) == 1 and call(bias=258) == 1 and call(idx=odd) == 1 and call(w=odd) == 1


def test_linear_refusals_on_the_host(lib):
    L = lib.load()
    p, null, odd = ctypes.c_void_p(256), None, ctypes.c_void_p(264)
    need = L.moe_linear_workspace_size()
    assert need >= lib.LINEAR_WORKSPACE_ZEROS and need % 256 == 0

    def call(R=4, K=64, N=64, G=2, dtype=0, a=p, a_stride=64, off=p, w=p, layout=0, bias=256, bias_dtype=2, act=1,
             res=256, res_stride=64, out_dtype=0, out=p, out_stride=64, ws=ctypes.c_void_p(4096), n=need):
        e = lib.Epilogue(bias, bias_dtype, act, res, res_stride)
        return L.moe_linear(R, K, N, G, dtype, a, a_stride, off, w, layout, ctypes.byref(e), out_dtype, out, out_stride,
                            ws, n, null)

    assert call(R=0, a=null, w=null, out=null) == 0
    assert call(R=-1) == 1 and call(K=0) == 1 and call(N=0) == 1 and call(G=0) == 1
    assert call(off=null) == 1                       # two groups need offsets
    assert call(layout=2) == 1 and call(act=5) == 1 and call(act=-1) == 1
    assert call(K=60) == 2 and call(N=60) == 2 and call(G=257) == 2 and call(R=1 << 31) == 2
    assert call(dtype=2) == 2 and call(dtype=9) == 2 and call(out_dtype=1) == 2 and call(bias_dtype=1) == 2
    assert call(R=(1 << 31) - 300, N=1 << 15, out_stride=1 << 15, res_stride=1 << 15) == 2
    assert call(ws=null) == 3 and call(ws=ctypes.c_void_p(4096 + 16)) == 3 and call(n=need - 1) == 3
    assert call(a=null) == 1 and call(w=null) == 1 and call(out=null) == 1 and call(a=odd) == 1 and call(w=odd) == 1
    assert call(a_stride=63) == 1 and call(a_stride=68) == 1 and call(out_stride=63) == 1 and call(res_stride=63) == 1
    assert call(out=ctypes.c_void_p(257)) == 1 and call(res=257) == 1 and call(bias=258) == 1
    assert call(off=ctypes.c_void_p(258)) == 1


def test_combine_refusals_on_the_host(lib):
    L = lib.load()
    p, null, odd = ctypes.c_void_p(256), None, ctypes.c_void_p(264)

    def call(T=4, H=64, k=2, R=8, dtype=0, y=p, ys=64, inv=p, w=p, out_dtype=0, res=p, rs=64, out=p, os=64):
        return L.moe_combine_rows(T, H, k, R, dtype, y, ys, inv, w, out_dtype, res, rs, out, os, null)

    assert call(T=0, y=null, inv=null, w=null, out=null) == 0
    assert call(T=-1) == 1 and call(H=0) == 1 and call(k=0) == 1 and call(R=-1) == 1
    assert call(H=60) == 2 and call(k=9) == 2 and call(dtype=3) == 2 and call(out_dtype=3) == 2
    assert call(T=1 << 30) == 2 and call(R=1 << 31) == 2 and call(T=1 << 62, k=4) == 2 and call(T=1 << 20, k=1, H=1 << 22) == 2
    assert call(y=null) == 1 and call(inv=null) == 1 and call(w=null) == 1 and call(out=null) == 1
    assert call(y=odd) == 1 and call(res=odd) == 1 and call(out=odd) == 1 and call(inv=ctypes.c_void_p(258)) == 1
    assert call(ys=63) == 1 and call(ys=68) == 1 and call(rs=56) == 1 and call(os=56) == 1


def test_binding_checks_tensors(lib):
    """Wrong shapes, types and layouts are refused by the binding (on CPU
    tensors: nothing reaches the library)."""
    bf = torch.bfloat16
    logits, bias = torch.zeros(4, 64), torch.zeros(64)
    a, w, off = torch.zeros(4, 64, dtype=bf), torch.zeros(2, 64, 32, dtype=bf), torch.zeros(3, dtype=torch.int32)
    b, ws = torch.zeros(2, 32), torch.zeros(256, dtype=torch.uint8)
    y, inv, tw = torch.zeros(8, 64, dtype=bf), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    bad = [
        lambda: lib.route_logits(logits.int(), 2),
        lambda: lib.route_logits(logits[0], 2),
        lambda: lib.route_logits(logits.t(), 2),
        lambda: lib.route_logits(logits, 2, scores="relu"),
        lambda: lib.route_logits(logits, 2, bias=bias[:32]),
        lambda: lib.route_logits(logits, 2, bias=bias.double()),
        lambda: lib.route_logits(logits, 2, topk_idx=torch.zeros(4, 2, dtype=torch.int64)),
        lambda: lib.route_logits(logits, 2, topk_w=torch.zeros(4, 3)),
        lambda: lib.route_logits(logits, 1 << 40),
        lambda: lib.route_logits(logits, 2),                                  # right, but not on a GPU
        lambda: lib.route_logits(None, 2),
        lambda: lib.linear(a.float(), w, ws, offsets=off),
        lambda: lib.linear(a, w.half(), ws, offsets=off),
        lambda: lib.linear(a, w[:, :32], ws, offsets=off),
        lambda: lib.linear(a, w[:, :, ::2], ws, offsets=off),
        lambda: lib.linear(a, w[0], ws),
        lambda: lib.linear(a.t(), w, ws, offsets=off),
        lambda: lib.linear(a, w, ws, offsets=off[:2]),
        lambda: lib.linear(a, w, ws, offsets=off.long()),
        lambda: lib.linear(a, w, ws, bias=b[:, :16], offsets=off),
        lambda: lib.linear(a, w, ws, bias=b.half(), offsets=off),
        lambda: lib.linear(a, w, ws, activation="tanh", offsets=off),
        lambda: lib.linear(a, w, ws, residual=torch.zeros(4, 32), offsets=off),
        lambda: lib.linear(a, w, ws, out_dtype=torch.float16, offsets=off),
        lambda: lib.linear(a, w, ws, out=torch.zeros(4, 32), offsets=off),
        lambda: lib.linear(a, w, ws.int(), offsets=off),
        lambda: lib.linear(a, w, ws, offsets=off),                            # right, but not on a GPU
        lambda: lib.combine_rows(y.int(), inv, tw),
        lambda: lib.combine_rows(y, inv[:3], tw),
        lambda: lib.combine_rows(y, inv.long(), tw),
        lambda: lib.combine_rows(y, inv, tw.half()),
        lambda: lib.combine_rows(y, inv, tw, residual=torch.zeros(4, 64)),
        lambda: lib.combine_rows(y, inv, tw, out_dtype=torch.int32),
        lambda: lib.combine_rows(y, inv, tw, out=torch.zeros(4, 64)),
        lambda: lib.combine_rows(y.t(), inv, tw),
        lambda: lib.combine_rows(y, inv, tw),                                 # right, but not on a GPU
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")


# ----------------------------------------------------------- route_logits --

def route64(logits, k, scores="softmax", bias=None, groups=1, top_groups=1, group_top=1, renormalize=False, scale=1.0):
    """The definition in 64 bits: (ids, weights)."""
    x = logits.double()
    T, E = x.shape
    if scores == "softmax":
        m = x.amax(1, keepdim=True)
        e = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
        s = e / e.sum(1, keepdim=True)
        s = torch.where(m == -math.inf, 0.0, s)
    else:
        s = 1 / (1 + torch.exp(-x))
    key = x if bias is None else s + bias.double()
    both = s if bias is None else key
    key, both = (torch.where(v.isnan(), -math.inf, v) for v in (key, both))
    kept = torch.ones(T, E, dtype=torch.bool, device=x.device)
    if groups > 1:
        part = (key if group_top == 1 else both).unflatten(1, (groups, -1))
        value = part.sort(dim=-1, descending=True).values[..., :group_top].sum(-1)
        place = value.sort(dim=-1, descending=True, stable=True).indices.argsort(-1)
        kept = (place < top_groups).repeat_interleave(E // groups, 1)
    # those kept first, each by its key, ties by index
    by_key = key.sort(dim=-1, descending=True, stable=True).indices
    first = kept.gather(1, by_key).int().sort(dim=-1, descending=True, stable=True).indices
    ids = by_key.gather(1, first)[:, :k]
    w = s.gather(1, ids)
    if renormalize:
        total = w.sum(1, keepdim=True)
        w = torch.where(total == 0, 0.0, w / total)
    w = torch.where(x.isnan().any(1, keepdim=True), math.nan, w * scale)
    return ids.int(), w


def check_route(got, want):
    ids, w = got
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    assert torch.equal(ids, want[0])
    nan = want[1].isnan()
    assert torch.equal(w.isnan(), nan)
    err = (w.double() - want[1]).abs()
    assert bool((err <= want[1].abs() * WEIGHT_TOL + 1e-37)[~nan].all())


ROUTES = [   # T, E, k, groups, top_groups, group_top
    (1, 1, 1, 1, 1, 1), (1, 64, 6, 1, 1, 1), (3, 8, 2, 1, 1, 1), (5, 8, 8, 1, 1, 1), (4097, 64, 6, 1, 1, 1),
    (100, 33, 8, 1, 1, 1), (77, 256, 8, 1, 1, 1), (513, 256, 8, 8, 4, 2), (300, 160, 6, 8, 3, 1), (64, 60, 4, 1, 1, 1),
    (65, 255, 8, 17, 3, 2), (65, 255, 7, 3, 2, 2), (65, 255, 8, 5, 1, 1), (65, 252, 8, 9, 2, 2), (65, 248, 8, 31, 1, 2),
    (65, 256, 8, 32, 32, 1), (65, 64, 8, 32, 4, 2), (65, 64, 2, 32, 1, 1), (40000, 128, 8, 4, 2, 2), (65, 32, 1, 32, 1, 1),
    (65, 32, 8, 32, 9, 1), (33, 14, 7, 2, 1, 1), (20000, 16, 4, 1, 1, 1), (65, 96, 8, 6, 3, 2),
]


@gpu
@pytest.mark.parametrize("T,E,k,groups,top_groups,group_top", ROUTES)
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_route(lib, T, E, k, groups, top_groups, group_top, dtype, scores):
    g = gen(T * E + k)
    logits = (2 * randn(g, T, E)).to(DTYPES[dtype])
    bias = (0.1 if scores == "sigmoid" else 0.5 / E) * randn(g, E)
    for b, renorm, scale in ((None, True, 1.0), (bias, True, 2.5), (bias, False, 1.0), (torch.zeros_like(bias), False, 16.0)):
        opts = dict(scores=scores, bias=b, groups=groups, top_groups=top_groups, group_top=group_top, renormalize=renorm,
                    scale=scale)
        check_route(lib.route_logits(logits, k, **opts), route64(logits, k, **opts))


@gpu
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top_groups,group_top", [(1, 1, 1), (8, 3, 1), (8, 3, 2)])
def test_route_near_and_equal_keys(lib, scores, groups, top_groups, group_top):
    """Keys that fp32 does not tell apart, and keys that are equal: many experts
    with the same few logits, biases that make scores differ by 2^-30 and less."""
    g = gen(11)
    T, E, k = 512, 128, 8
    logits = torch.randint(0, 3, (T, E), generator=g, device="cuda").float() * 0.5
    s = 1 / (1 + torch.exp(-logits.double())) if scores == "sigmoid" else torch.softmax(logits.double(), 1)
    near = (0.75 - s).float()                      # per token: here of token 0
    steps = torch.randint(0, 3, (E,), generator=g, device="cuda") * 2.0 ** -26
    for bias in (torch.zeros(E, device="cuda"), near[0], near[0] + steps, steps.float()):
        opts = dict(scores=scores, bias=bias.contiguous(), groups=groups, top_groups=top_groups, group_top=group_top)
        rows = logits.clone()
        rows[::2] = logits[0]                      # all of token 0's keys about 0.75
        check_route(lib.route_logits(rows, k, **opts), route64(rows, k, **opts))
    # logits a step of fp32 apart
    rows = 1 + torch.randint(0, 5, (T, E), generator=g, device="cuda").float() * 2.0 ** -23
    bias = torch.randint(0, 2, (E,), generator=g, device="cuda").float() * 2.0 ** -24
    for b in (None, bias):
        opts = dict(scores=scores, bias=b, groups=groups, top_groups=top_groups, group_top=group_top)
        check_route(lib.route_logits(rows, k, **opts), route64(rows, k, **opts))


@gpu
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("groups,top_groups,group_top", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
def test_route_masked_and_special_rows(lib, scores, bias, groups, top_groups, group_top):
    """Logits of -inf (a few, all but one, all), the types' lowest value, NaN, far
    apart and tiny scores; biases of -inf."""
    g = gen(5)
    E, k = 32, 6
    x = randn(g, 12, E)
    x[0, ::3] = -math.inf
    x[1] = -math.inf
    x[2, 1:] = -math.inf
    x[3] = torch.finfo(torch.float32).min
    x[4, 5:] = torch.finfo(torch.float32).min
    x[5, 7] = math.nan
    x[6] = math.nan
    x[7] = torch.linspace(-300, 300, E, device="cuda")
    x[8] = torch.linspace(-95, -90, E, device="cuda")
    x[9] = 0.0
    x[9, ::2] = -0.0
    b = 0.01 * randn(g, E) if bias else None
    if bias:
        b[3] = b[17] = -math.inf
    for renorm in (False, True):
        opts = dict(scores=scores, bias=b, groups=groups, top_groups=top_groups, group_top=group_top, renormalize=renorm)
        ids, w = lib.route_logits(x, k, **opts)
        want_ids, want_w = route64(x, k, **opts)
        assert torch.equal(ids, want_ids)
        nan = want_w.isnan()
        assert torch.equal(w.isnan(), nan)
        # e^x and the exponents of logits up to 300 apart
        assert bool(((w.double() - want_w).abs() <= want_w.abs() * 200 * 2.0 ** -23 + 1e-28)[~nan].all())
        assert bool((w[1] == 0).all())
    # +inf: a sigmoid of 1; a softmax of inf - inf
    y = randn(g, 3, E)
    y[1, 9] = math.inf
    ids, w = lib.route_logits(y, k, scores=scores)
    assert ids[1, 0] == 9 and bool((ids >= 0).all()) and bool((ids < E).all())
    assert float(w[1, 0]) == 1.0 if scores == "sigmoid" else bool(w[1].isnan().any())
    assert bool(w[[0, 2]].isfinite().all())


@gpu
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_route_equal_rows(lib, scores):
    """Rows of equal logits (a router before its training), more experts than a warp lists."""
    x = torch.zeros(3000, 256, device="cuda")
    for opts in (dict(), dict(bias=torch.zeros(256, device="cuda")), dict(groups=8, top_groups=3, group_top=2),
                 dict(groups=8, top_groups=3), dict(renormalize=True, groups=4, top_groups=1)):
        opts["scores"] = scores
        check_route(lib.route_logits(x, 8, **opts), route64(x, 8, **opts))


@gpu
def test_route_on_a_side_stream(lib):
    g = gen(21)
    x = randn(g, 4000, 128)
    want = lib.route_logits(x, 8, scores="sigmoid", renormalize=True)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        y = x * 1.0
    got = lib.route_logits(y, 8, scores="sigmoid", renormalize=True, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@gpu
def test_route_strides_outputs_and_empty(lib):
    g = gen(3)
    wide = randn(g, 50, 200)
    for dtype in DTYPES.values():
        v = wide.to(dtype)
        for view in (v[:, 3:67], v[:, 64:128], v[::2, 1:65], v[:1, :64]):
            check_route(lib.route_logits(view, 6, renormalize=True), route64(view, 6, renormalize=True))
    idx, w = torch.empty(50, 4, dtype=torch.int32, device="cuda"), torch.empty(50, 4, device="cuda")
    got = lib.route_logits(wide, 4, topk_idx=idx, topk_w=w)
    assert got[0].data_ptr() == idx.data_ptr() and got[1].data_ptr() == w.data_ptr()
    check_route((idx, w), route64(wide, 4))
    # the two outputs of a call are apart, and either may outlive the other
    ids, weights = lib.route_logits(wide, 4)
    assert ids.is_contiguous() and weights.is_contiguous() and ids.shape == weights.shape == (50, 4)
    want = weights.clone()
    ids.fill_(-1)
    assert torch.equal(weights, want) and torch.equal(w, want)
    del ids
    torch.full((400,), 7, dtype=torch.int32, device="cuda")
    assert torch.equal(weights, want) and torch.equal(weights + 0, want) and bool((weights.sum(0) > 0).all())
    got = lib.route_logits(wide[:0], 4)
    assert got[0].shape == (0, 4) and got[1].shape == (0, 4)
    for bad in (dict(k=9), dict(k=0), dict(k=4, groups=7), dict(k=4, top_groups=2), dict(k=4, group_top=3)):
        with pytest.raises(lib.MoeError):
            lib.route_logits(wide, **bad)


@gpu
def test_route_matches_route(lib):
    """Softmax, renormalized, on the logits of x and Wg: what route() selects."""
    g = gen(8)
    T, H, E, k = 1000, 256, 64, 6
    x, Wg = randn(g, T, H).bfloat16(), (0.1 * randn(g, H, E)).bfloat16()
    d = lib.make_dims(T, H, 64, E, k)
    ids, w = lib.route(d, x, Wg)
    logits = x.double() @ Wg.double()
    top = logits.sort(dim=-1, descending=True).values
    clear = ((top[:, :k] - top[:, 1: k + 1]) > 1e-4).all(1)
    got, gw = lib.route_logits(logits.float(), k, renormalize=True)
    assert bool(clear.sum() > 900)
    assert torch.equal(got[clear], ids[clear])
    assert bool(((gw - w)[clear].abs() <= 1e-4).all())


# ----------------------------------------------------------------- linear --

def act64(name, v):
    if name == "relu":
        return torch.where(v < 0, 0.0, v)
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return v * 0.5 * torch.erfc(-v / math.sqrt(2))
    if name == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def linear64(a, w, ends, bias=None, act=None, residual=None):
    """(out, sum of the terms' magnitudes) in 64 bits, NaN in rows of no group."""
    out = torch.full((a.shape[0], w.shape[2]), math.nan, dtype=torch.float64, device="cuda")
    mag = out.clone()
    for g in range(w.shape[0]):
        lo, hi = ends[g], ends[g + 1]
        if hi > lo:
            v, m = a[lo:hi].double() @ w[g].double(), a[lo:hi].double().abs() @ w[g].double().abs()
            if bias is not None:
                v, m = v + bias[g].double(), m + bias[g].double().abs()
            v = act64(act, v)
            if residual is not None:
                v, m = v + residual[lo:hi].double(), m + residual[lo:hi].double().abs()
            out[lo:hi], mag[lo:hi] = v, m
    return out, mag


def check_linear(out, ref, mag, K):
    half = torch.finfo(out.dtype).eps / 2
    tiny = torch.finfo(out.dtype).tiny * half if out.dtype == torch.float16 else 0.0
    rows = ~ref[:, 0].isnan()
    out, ref, mag = out[rows].double(), ref[rows], mag[rows]
    assert bool(((out - ref).abs() <= ref.abs() * half + mag * ((K + 64) * 1.13 * 2.0 ** -23 + 2.0 ** -20) + tiny).all())
    # over all values: the tensor cores' sums of 512 products (2048 for 16-bit outputs), 16
    # at a time, each off by a step at most, before they are added up in fp32, and an
    # activation's own error
    rel = float((out - ref).norm() / ref.norm())
    assert rel <= half + (32 if half < 2.0 ** -20 else 128) * 2.0 ** -23 + 2.0 ** -20, rel


def offsets_of(counts, first=0):
    o = [first]
    for c in counts:
        o.append(o[-1] + c)
    return torch.tensor(o, dtype=torch.int32, device="cuda"), o


def weight(g, G, K, N, dtype, layout):
    w = K ** -0.5 * randn(g, G, K, N)
    return w.to(dtype) if layout == "kn" else w.transpose(1, 2).contiguous().to(dtype).transpose(1, 2)


LINEARS = [   # K, N, rows of each group
    (8, 8, [1]), (64, 8, [0, 1, 0]), (40, 72, [5]), (128, 128, [128]), (136, 136, [3, 0, 130]), (256, 256, [129, 1]),
    (2048, 264, [0, 0, 7]), (1408, 2048, [1] * 6 + [0] * 10), (400, 400, [127, 128, 129, 0, 300]), (4096, 1024, [1]),
    (4096, 1024, [40]), (14336, 256, [1, 0, 1]), (14336, 256, [2, 128, 1]), (20480, 384, [333]),
    (2048, 1408, [90 + (7 * i) % 13 for i in range(64)]), (512, 128, [1] * 256), (256, 512, [3] * 255 + [1000]),
    (256, 320, [2085]), (400, 272, [5000, 0, 5001, 100]), (4096, 14336, [1, 1]), (2048, 40960, [17]), (16384, 512, [1]),
    (8192, 272, [130]), (8192, 144, [20, 40, 0, 33]), (1024, 2064, [1]), (520, 264, [257, 255, 16, 17, 512, 513]),
    (576, 4096, [4600]), (64, 64, [20000]), (4096, 256, [2048]), (4160, 4096, [900]),
    (4096, 128, [4500]), (20480, 128, [3900]), (320, 2048, [700, 1, 900]), (14336, 2048, [1000]), (1024, 256, [97]), (4096, 512, [31, 33, 64, 65]),
]


@gpu
@pytest.mark.parametrize("K,N,counts", LINEARS, ids=lambda v: str(v) if isinstance(v, int) else f"{len(v)}g{sum(v)}r")
@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16")])
@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_linear(lib, ws, K, N, counts, dtype, out_dtype, layout):
    g = gen(K * N + sum(counts))
    R, dt, od = sum(counts), DTYPES[dtype], DTYPES[out_dtype]
    a, w = randn(g, R, K).to(dt), weight(g, len(counts), K, N, dt, layout)
    off, ends = offsets_of(counts)
    out = torch.full((R, N), math.nan, dtype=od, device="cuda")
    lib.linear(a, w, ws, offsets=off, out_dtype=od, out=out)
    assert lib.check(ws) == lib.MOE_OK
    check_linear(out, *linear64(a, w, ends), K)
    assert torch.equal(out, lib.linear(a, w, ws, offsets=off, out_dtype=od))
    if len(counts) == 1:
        assert torch.equal(out, lib.linear(a, w, ws, out_dtype=od))
    # the whole epilogue on the same operands
    bias, res = randn(g, len(counts), N), randn(g, R, N).to(od)
    out = lib.linear(a, w, ws, bias=bias, activation="gelu", residual=res, offsets=off, out_dtype=od)
    assert lib.check(ws) == lib.MOE_OK
    check_linear(out, *linear64(a, w, ends, bias, "gelu", res), K)


def test_linear_forms(lib):
    """The form of each size, and sizes that have none."""
    few, one, pair, half = lib.LINEAR_FORM_FEW, lib.LINEAR_FORM_ONE, lib.LINEAR_FORM_PAIR, lib.LINEAR_FORM_PAIR_HALF
    for (R, K, N, G), want in {(1, 4096, 14336, 1): few, (16, 64, 64, 1): few, (17, 64, 64, 1): half, (1, 64, 64, 2): one,
                               (100, 4096, 4096, 1): half, (8192, 4096, 256, 1): half, (20000, 4096, 128, 1): one,
                               (768, 2048, 1408, 64): one, (8192, 4096, 4096, 1): pair, (160, 4096, 14336, 1): pair,
                               (16384, 4096, 14336, 8): pair, (20000, 2048, 1408, 64): pair}.items():
        assert lib.linear_form_selftest(R, K, N, G) == want, (R, K, N, G)
    for R, K, N, G in (0, 64, 64, 1), (4, 60, 64, 1), (4, 64, 4, 1), (4, 64, 64, 257), (4, 0, 64, 1), (-1, 64, 64, 1):
        assert lib.linear_form_selftest(R, K, N, G) == -1
    assert lib.linear_form_selftest(4, 64, 64, 1, num_sms=0) == -1
    assert lib.linear_form_selftest(8192, 4096, 4096, 1, num_sms=1) == one      # no SM for a pair's second CTA
    forms = {lib.linear_form_selftest(max(1, sum(c)), K, N, len(c)) for K, N, c in LINEARS}
    assert forms == {few, one, pair, half}                                    # what test_linear runs


@gpu
@pytest.mark.parametrize("R,K,N", [(1, 2048, 2048), (300, 4096, 512), (2048, 1024, 4096), (20000, 1024, 128)])
def test_linear_captured_beside_eager(lib, R, K, N):
    """Each form captured and replayed on new inputs, with eager calls of another form and
    of the same one between the replays (their workspace is another)."""
    g = gen(R)
    a, other = randn(g, R, K).bfloat16(), randn(g, R, K).bfloat16()
    w, bias = weight(g, 1, K, N, torch.bfloat16, "kn"), randn(g, 1, N)
    ws, graph_ws = lib.linear_workspace(), lib.linear_workspace()
    want = [lib.linear(x, w, ws, bias=bias, activation="silu") for x in (a, other)]
    x = a.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        lib.linear(x, w, graph_ws, bias=bias, activation="silu")
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = lib.linear(x, w, graph_ws, bias=bias, activation="silu")
        second = lib.linear(x, w, graph_ws, bias=bias, activation="silu", out_dtype=torch.float32)
    for rows, ref in ((other, want[1]), (a, want[0])):
        x.copy_(rows)
        graph.replay()
        eager = lib.linear(a, w, ws, bias=bias, activation="silu")
        lib.linear(a[:3], w, ws)
        assert torch.equal(first, ref) and torch.equal(eager, want[0])
        # (the fp32 sum differs from the one that was rounded by both sums' own errors, which are
        # of the terms' magnitude, so it is held to the definition instead)
        check_linear(second, *linear64(rows, w, [0, R], bias, "silu"), K)
    assert lib.check(ws) == lib.MOE_OK and lib.check(graph_ws) == lib.MOE_OK


@gpu
def test_linear_workspace_of_every_form(lib, ws):
    """One workspace for products of all forms and sizes, one after another, on two
    streams in turn."""
    g = gen(12)
    jobs = []
    for R, K, N, G in ((3, 8192, 512, 1), (900, 4160, 512, 1), (40, 2048, 264, 8), (3000, 512, 1024, 3), (1, 512, 128, 1)):
        a, w = randn(g, R, K).bfloat16(), weight(g, G, K, N, torch.bfloat16, "nk")
        off, _ = offsets_of([R // G] * (G - 1) + [R - R // G * (G - 1)])
        jobs.append((a, w, off, lib.linear(a, w, ws, offsets=off).clone()))
    side = torch.cuda.Stream()
    for i, (a, w, off, want) in enumerate(jobs * 3):
        stream = side if i % 2 else None
        here = stream or torch.cuda.current_stream()
        here.wait_stream(torch.cuda.current_stream() if stream else side)
        got = lib.linear(a, w, ws, offsets=off, stream=stream)
        here.synchronize()
        assert torch.equal(got, want)
    assert lib.check(ws) == lib.MOE_OK


@gpu
def test_linear_activations_of_extremes(lib, ws):
    """Sums of infinity and of the largest magnitudes, through the bias."""
    a = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(1, 64, 64, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(1, 64, device="cuda")
    x[0, :8] = torch.tensor([math.inf, 1e38, 1e20, 300.0, -300.0, -1e20, -1e38, math.nan])
    for act in ("relu", "silu", "gelu", "gelu_tanh"):
        y = lib.linear(a, w, ws, bias=x, activation=act, out_dtype=torch.float32)
        assert torch.equal(y[0, :4], x[0, :4]), act
        assert bool((y[0, 4:7] == 0).all()) and bool(y[0, 7].isnan()) and bool((y[0, 8:] == 0).all()), act


@gpu
@pytest.mark.parametrize("act", [None, "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("out_dtype", ["bf16", "fp16", "fp32"])
def test_linear_epilogue(lib, ws, act, out_dtype):
    """Each activation with biases of both types, and a residual, over arguments from
    far below to far above zero."""
    g = gen(9)
    counts = [37, 0, 150, 13]
    R, K, N, od = sum(counts), 320, 200, DTYPES[out_dtype]
    dt = torch.float16 if out_dtype == "fp16" else torch.bfloat16
    off, ends = offsets_of(counts)
    a, w = (4 * randn(g, R, K)).to(dt), weight(g, 4, K, N, dt, "kn")
    for bias in (None, 3 * randn(g, 4, N), (3 * randn(g, 4, N)).to(dt)):
        for res in (None, randn(g, R, N).to(od)):
            out = lib.linear(a, w, ws, bias=bias, activation=act, residual=res, offsets=off, out_dtype=od)
            check_linear(out, *linear64(a, w, ends, bias, act, res), K)
    assert lib.check(ws) == lib.MOE_OK


@gpu
def test_linear_strides_and_in_place(lib, ws):
    g = gen(2)
    R, K, N = 70, 200, 136
    wide = randn(g, R, 512).bfloat16()
    a, w = wide[:, 8:208], weight(g, 1, K, N, torch.bfloat16, "kn")
    bias, res = randn(g, 1, N), randn(g, R, N).bfloat16()
    want = lib.linear(a.contiguous(), w, ws, bias=bias, activation="silu", residual=res)
    # the residual and the output in one memory, its rows an odd number of elements apart
    mem = torch.full((R, 301), 7.0, dtype=torch.bfloat16, device="cuda")
    view = mem[:, 5:5 + N]
    view.copy_(res)
    got = lib.linear(a, w, ws, bias=bias, activation="silu", residual=view, out=view)
    assert got.data_ptr() == view.data_ptr() and torch.equal(got, want)
    assert bool((mem[:, :5] == 7).all()) and bool((mem[:, 5 + N:] == 7).all())
    with pytest.raises(lib.MoeError):
        lib.linear(wide[:, 4:204], w, ws)     # rows start 8 bytes off a 16-byte boundary
    one = lib.linear(wide[:1, 8:208], w, ws, bias=bias, activation="silu", residual=res[:1])
    assert torch.equal(one, want[:1]) or bool(((one - want[:1]).abs() <= want[:1].abs() * 2.0 ** -7).all())


@gpu
def test_linear_rows_outside_groups_and_bad_offsets(lib, ws):
    g = gen(3)
    K, N, R = 256, 320, 50
    a, w = randn(g, R, K).bfloat16(), weight(g, 3, K, N, torch.bfloat16, "kn")
    off, ends = offsets_of([10, 0, 20], first=5)
    out = torch.full((R, N), -7.0, dtype=torch.float32, device="cuda")
    lib.linear(a, w, ws, offsets=off, out_dtype=torch.float32, out=out)
    assert lib.check(ws) == lib.MOE_OK
    assert bool((out[:5] == -7).all()) and bool((out[35:] == -7).all())
    check_linear(out, *linear64(a, w, ends), K)
    for bad, status in ([0, 0, 0, 0], 0), ([0, 30, 20, 50], 6), ([0, 10, 20, 51], 6), ([-1, 10, 20, 30], 6):
        out.fill_(-7.0)
        o = torch.tensor(bad, dtype=torch.int32, device="cuda")
        lib.linear(a, w, ws, offsets=o, out_dtype=torch.float32, out=out)
        assert lib.check(ws) == status
        assert bool((out == -7).all())
    assert lib.linear(a[:0], w, ws, offsets=off).shape == (0, N)


@gpu
@pytest.mark.parametrize("R", [20, 700])
def test_linear_nan_stays_in_its_row(lib, ws, R):
    g = gen(4)
    K, N = 520, 256
    a, w = randn(g, R, K).bfloat16(), weight(g, 1, K, N, torch.bfloat16, "nk")
    for act in (None, "relu"):
        want = lib.linear(a, w, ws, activation=act, out_dtype=torch.float32)
        b = a.clone()
        b[3, 100] = math.nan
        b[7, 519] = math.inf
        got = lib.linear(b, w, ws, activation=act, out_dtype=torch.float32)
        assert bool(got[3].isnan().all()) and (act == "relu" or not bool(got[7].isfinite().any()))
        rows = [i for i in range(R) if i not in (3, 7)]
        assert torch.equal(got[rows], want[rows])


@gpu
def test_linear_long_output(lib, ws):
    """An output of more elements than 32 bits count."""
    g = gen(6)
    R, K, N = 140001, 64, 16384
    a, w = randn(g, R, K).bfloat16(), weight(g, 2, K, N, torch.bfloat16, "kn")
    off = torch.tensor([0, 139000, R], dtype=torch.int32, device="cuda")
    out = lib.linear(a, w, ws, offsets=off)
    assert lib.check(ws) == lib.MOE_OK
    for lo, e in ((0, 0), (138990, 0), (R - 10, 1)):
        x, y = a[lo: lo + 10].double(), w[e].double()
        check_linear(out[lo: lo + 10], x @ y, x.abs() @ y.abs(), K)


# ----------------------------------------------------------- combine_rows --

def combine64(y, inv, w, residual):
    """(out, sum of the terms' magnitudes) in 64 bits."""
    T, k = w.shape
    at = inv.view(T, k).long()
    out = torch.zeros(T, y.shape[1], dtype=torch.float64, device="cuda")
    mag = out.clone()
    for j in range(k):
        there = ((at[:, j] >= 0) & (at[:, j] < y.shape[0])).nonzero().flatten()
        v = w[there, j, None].double() * y[at[there, j]].double()
        out[there] += v
        mag[there] += v.abs()
    if residual is not None:
        out, mag = out + residual.double(), mag + residual.double().abs()
    return out, mag


def check_combine(out, ref, mag):
    half = torch.finfo(out.dtype).eps / 2
    tiny = torch.finfo(out.dtype).tiny * half if out.dtype == torch.float16 else 0.0
    assert bool(((out.double() - ref).abs() <= ref.abs() * half + mag * 12 * 2.0 ** -24 + tiny).all())


@gpu
@pytest.mark.parametrize("T,H,k", [(1, 8, 1), (1, 4096, 2), (3, 64, 8), (7, 1032, 5), (129, 2048, 6), (33, 3584, 8),
                                   (2, 16384, 3), (5000, 136, 4), (70000, 8, 1)])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("out_dtype", list(DTYPES))
def test_combine(lib, T, H, k, dtype, out_dtype):
    g = gen(T + H + k)
    R = T * k
    y, w = randn(g, R, H).to(DTYPES[dtype]), torch.softmax(randn(g, T, k), -1)
    inv = torch.randperm(R, generator=g, device="cuda").int()
    res = randn(g, T, H).to(DTYPES[out_dtype])
    for r in (None, res):
        out = lib.combine_rows(y, inv, w, residual=r, out_dtype=DTYPES[out_dtype])
        check_combine(out, *combine64(y, inv, w, r))
    # dropped assignments (also all of a token's) and rows used twice
    inv = torch.randint(-2, R + 2, (T, k), generator=g, device="cuda").int()
    inv[0] = -1
    out = lib.combine_rows(y, inv, w, residual=res, out_dtype=DTYPES[out_dtype])
    check_combine(out, *combine64(y, inv, w, res))
    assert torch.equal(out[0], res[0])


@gpu
def test_combine_strides_in_place_and_empty(lib):
    g = gen(7)
    T, H, k = 40, 256, 3
    wide = randn(g, T * k, 640).bfloat16()
    inv, w = torch.randperm(T * k, generator=g, device="cuda").int(), torch.rand(T, k, generator=g, device="cuda")
    mem = randn(g, T, 512)
    res = mem[:, 128:384]
    keep = mem.clone()
    want = lib.combine_rows(wide[:, 64:320].contiguous(), inv, w, residual=res.contiguous(), out_dtype=torch.float32)
    got = lib.combine_rows(wide[:, 64:320], inv, w, residual=res, out_dtype=torch.float32, out=res)
    assert torch.equal(got, want) and torch.equal(mem[:, 128:384], want)
    assert torch.equal(mem[:, :128], keep[:, :128]) and torch.equal(mem[:, 384:], keep[:, 384:])
    # a NaN in a row that nothing points to stays there; no rows at all
    y = wide[:, :H].contiguous()
    inv[inv == 5] = -1
    want = lib.combine_rows(y, inv, w)
    y[5] = math.nan
    assert torch.equal(lib.combine_rows(y, inv, w), want)
    none = lib.combine_rows(y[:0], torch.full_like(inv, -1), w)
    assert bool((none == 0).all())
    assert lib.combine_rows(y, inv[:0], w[:0]).shape == (0, H)
    with pytest.raises(lib.MoeError):
        lib.combine_rows(wide[:, 4:260], inv, w)


@gpu
def test_combine_long(lib):
    """Rows of more elements than 32 bits count."""
    R, H, T = 300000, 8192, 4
    y = torch.zeros(R, H, dtype=torch.bfloat16, device="cuda")
    y[-1] = 3
    y[0] = 1
    inv = torch.tensor([R - 1, 0, R - 1, R - 1, 0, 0, -1, R], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.25]], device="cuda").expand(T, 2).contiguous()
    out = lib.combine_rows(y, inv, w, out_dtype=torch.float32)
    assert out[:, 0].tolist() == [1.75, 2.25, 0.75, 0.0] and bool((out == out[:, :1]).all())


# --------------------------------------------------------------- together --

def chain(lib, x, Wg, gate_bias, w1, b1, w2, b2, k, ws, perm_ws, stream=None):
    """An expert layer with biased gelu experts behind a sigmoid router, added to x."""
    T, H = x.shape
    E = Wg.shape[2]
    d = lib.make_dims(T, H, 64, E, k)
    logits = lib.linear(x, Wg, ws, out_dtype=torch.float32, stream=stream)
    ids, w = lib.route_logits(logits, k, scores="sigmoid", bias=gate_bias, groups=4, top_groups=2, group_top=2,
                              renormalize=True, scale=2.5, stream=stream)
    _, offsets, _, inv_pos, rows = lib.permute(d, ids, perm_ws, x=x, want_x_perm=True, stream=stream)
    h = lib.linear(rows, w1, ws, bias=b1, activation="gelu", offsets=offsets, stream=stream)
    y = lib.linear(h, w2, ws, bias=b2, offsets=offsets, stream=stream)
    return logits, ids, w, h, y, lib.combine_rows(y, inv_pos, w, residual=x, stream=stream)


def chain_inputs(g, T, H=512, F=384, E=32):
    return (randn(g, T, H).bfloat16(), (0.1 * randn(g, 1, H, E)).bfloat16(), 0.05 * randn(g, E),
            (H ** -0.5 * randn(g, E, H, F)).bfloat16(), 0.3 * randn(g, E, F), (F ** -0.5 * randn(g, E, F, H)).bfloat16(),
            0.3 * randn(g, E, H))


@gpu
@pytest.mark.parametrize("T", [1, 37, 900])
def test_chain(lib, ws, T):
    """The operators together, each step's output from the last one's in 64 bits."""
    g = gen(T)
    k, E = 6, 32
    inp = chain_inputs(g, T)
    x, Wg, gb, w1, b1, w2, b2 = inp
    perm_ws = lib.workspace(lib.make_dims(T, 512, 64, E, k))
    logits, ids, w, h, y, out = chain(lib, *inp, k, ws, perm_ws)
    assert lib.check(ws) == lib.MOE_OK and lib.check(perm_ws) == lib.MOE_OK
    check_linear(logits, *linear64(x, Wg, [0, T]), 512)
    check_route((ids, w), route64(logits, k, scores="sigmoid", bias=gb, groups=4, top_groups=2, group_top=2,
                                  renormalize=True, scale=2.5))
    want = x.double()
    # the experts of each token, from its own row
    flat = ids.flatten().long()
    rows = x.repeat_interleave(k, 0)
    ref = torch.empty(T * k, 512, dtype=torch.float64, device="cuda")
    for e in flat.unique().tolist():
        at = (flat == e).nonzero().flatten()
        hid = act64("gelu", rows[at].double() @ w1[e].double() + b1[e].double())
        ref[at] = hid @ w2[e].double() + b2[e].double()
    want = want + (ref.view(T, k, -1) * w.double().unsqueeze(-1)).sum(1)
    # h and y are rounded to bf16 on the way, and the output: three half steps
    rel = float((out.double() - want).norm() / want.norm())
    assert rel <= 2.0 ** -8 * 3 ** 0.5, rel


@gpu
def test_chain_in_a_graph_on_a_side_stream(lib):
    """Captured and replayed on new inputs, beside eager calls with another workspace."""
    g = gen(77)
    T, k, E = 130, 6, 32
    inp, other = chain_inputs(g, T), randn(g, T, 512).bfloat16()
    ws, perm_ws = lib.linear_workspace(), lib.workspace(lib.make_dims(T, 512, 64, E, k))
    x = inp[0].clone()
    want = [t.clone() for t in chain(lib, *inp, k, ws, perm_ws)]
    want_other = [t.clone() for t in chain(lib, other, *inp[1:], k, ws, perm_ws)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = chain(lib, x, *inp[1:], k, ws, perm_ws, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph_ws, graph_perm = lib.linear_workspace(), lib.workspace(lib.make_dims(T, 512, 64, E, k))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(lib, x, *inp[1:], k, graph_ws, graph_perm)
    for rows, ref in ((inp[0], want), (other, want_other), (inp[0], want)):
        x.copy_(rows)
        graph.replay()
        eager = chain(lib, other, *inp[1:], k, ws, perm_ws)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
        assert all(torch.equal(a, b) for a, b in zip(eager, want_other))
    for w in (ws, graph_ws, perm_ws, graph_perm):
        assert lib.check(w) == lib.MOE_OK
