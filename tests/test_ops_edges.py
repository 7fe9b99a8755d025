"""What route_logits, linear and combine_rows promise beyond the definitions that
test_ops.py holds them to. Tolerances are derived where they stand, in steps of fp32
(2^-23 of a value; half of one for a rounding).
"""
import ctypes
import io
import math
import random

import pytest
import torch

from test_ops import DTYPES, act64, check_linear, check_route, gen, lib, linear64, offsets_of, randn, route64, weight, ws  # noqa: F401

gpu = pytest.mark.gpu


# ------------------------------------------------------------ linear: sums --

@gpu
@pytest.mark.parametrize("R,K,N,G", [(16, 4096, 28672, 1), (768, 2048, 1408, 64), (20000, 4096, 128, 1), (400, 4096, 8192, 1),
                                     (8192, 2048, 1024, 1), (4096, 14336, 512, 2), (300, 1032, 264, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("one_sign", [False, True])
def test_linear_rounds_the_fp32_output_once(lib, ws, R, K, N, G, dtype, one_sign):
    """An output of 16 bits is that of 32 bits, rounded: sums, bias, activation and residual are
    the same whatever the output's type. Bit for bit, on sums that cancel and on sums that
    only grow (where a longer run of the tensor cores, which round towards zero, drifts)."""
    g = gen(R + K)
    dt = DTYPES[dtype]
    off, _ = offsets_of([R // G] * G)
    a, w = randn(g, R, K), randn(g, G, N, K) * K ** -0.5
    if one_sign:
        a, w = a.abs(), w.abs()
    a, w = a.to(dt), w.to(dt).transpose(1, 2)
    bias, res = randn(g, G, N), randn(g, R, N).to(dt)
    for act, b, r in ((None, None, None), (None, bias, res), ("silu", bias, None), ("relu", None, res)):
        out = lib.linear(a, w, ws, bias=b, activation=act, residual=r, offsets=off)
        wide = lib.linear(a, w, ws, bias=b, activation=act, residual=None if r is None else r.float(), offsets=off,
                          out_dtype=torch.float32)
        assert lib.check(ws) == lib.MOE_OK
        assert torch.equal(out, wide.to(dt)), (act, int((out != wide.to(dt)).sum()), out.numel())


# ------------------------------------------------- route_logits: infinities --

@gpu
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("forced", [(5,), (5, 6), (30, 2), (1, 9, 17, 25), (0, 1, 2, 3, 4, 5, 6, 7)])
@pytest.mark.parametrize("groups,top_groups,group_top", [(1, 1, 1), (4, 2, 1), (4, 2, 2), (8, 1, 2)])
@pytest.mark.parametrize("T", [1, 301, 8192])
def test_route_forced_experts(lib, scores, forced, groups, top_groups, group_top, T):
    """A bias of +inf forces an expert in, by index among several; the others are ordered
    as ever, also where fp32 does not tell them apart."""
    g = gen(len(forced) + T)
    E, k = 32, 4
    few = torch.randint(0, 3, (T, E), generator=g, device="cuda").float() * 0.5
    near = (0.75 - (torch.sigmoid(few[0].double()) if scores == "sigmoid" else torch.softmax(few[0].double(), 0))).float()
    for x, bias in ((few, torch.zeros(E, device="cuda")), (few[:1].expand(T, E).contiguous(), near),
                    (randn(g, T, E), 0.01 * randn(g, E))):
        bias[list(forced)] = math.inf
        for drop in (False, True):
            if drop:
                bias[[10, 13, 20]] = -math.inf
            for renorm in (False, True):
                opts = dict(scores=scores, bias=bias, groups=groups, top_groups=top_groups, group_top=group_top,
                            renormalize=renorm)
                idx = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
                w = torch.full((T, k), math.nan, device="cuda")
                lib.route_logits(x, k, topk_idx=idx, topk_w=w, **opts)
                check_route((idx, w), route64(x, k, **opts))


# ---------------------------------------------------- route_logits: outputs --

@gpu
def test_route_outputs_can_be_stored(lib):
    """The two outputs are tensors of their own: stored together, and neither holds the
    other's memory."""
    x = randn(gen(1), 40, 64)
    ids, w = lib.route_logits(x, 6)
    for t in (ids, w):
        assert t.storage_offset() == 0 and t.untyped_storage().nbytes() == 40 * 6 * 4
    memory = io.BytesIO()
    torch.save({"ids": ids, "w": w}, memory)
    memory.seek(0)
    back = torch.load(memory)
    assert torch.equal(back["ids"], ids) and torch.equal(back["w"], w)


# ------------------------------------------------------- permute's row types --

def test_permute_refuses_other_rows(lib):
    """permute copies rows of 16-bit values as they are: others, of other sizes or not
    contiguous, are refused before anything is launched."""
    d = lib.make_dims(4, 64, 64, 8, 2)
    ids, x = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 64, dtype=torch.bfloat16)
    one = torch.zeros(256, dtype=torch.uint8)
    for bad in (x.float(), x.to(torch.int16), x[:3], x[:, :32], x.t(), torch.zeros(4, 128, dtype=torch.bfloat16)[:, ::2]):
        with pytest.raises(ValueError, match="^x:"):
            lib.permute(d, ids, one, x=bad, want_x_perm=True)
        with pytest.raises(ValueError, match="^x:"):
            lib.permute_static(d, ids, x=bad, want_x_perm=True)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_permute_keeps_the_rows_type(lib, dtype):
    T, H, E, k = 100, 128, 16, 3
    g = gen(4)
    d = lib.make_dims(T, H, 64, E, k)
    x = randn(g, T, H).to(DTYPES[dtype])
    ids = randn(g, T, E).topk(k, -1).indices.int()
    for got in (lib.permute(d, ids, lib.workspace(d), x=x, want_x_perm=True), lib.permute_static(d, ids, x=x, want_x_perm=True)):
        src, rows = got[2], got[4]
        # (row p is assignment src[p] = t k + j; indexed on the host)
        assert rows.dtype == x.dtype and torch.equal(rows.cpu(), x.cpu()[src.cpu().long() // k])
    # the rows in another shape, and the first of a longer buffer
    for y in (x.view(4, T // 4, H), torch.cat([x, x])):
        assert torch.equal(lib.permute(d, ids, lib.workspace(d), x=y, want_x_perm=True)[4], rows)


@gpu
@pytest.mark.parametrize("T", [1, 150])
def test_chain_in_fp16(lib, ws, T):
    """An expert layer on fp16 rows: router, dispatch, biased gelu experts, weighted sum."""
    g = gen(T)
    H, F, E, k = 256, 384, 16, 3
    d = lib.make_dims(T, H, 64, E, k)
    x, Wg = randn(g, T, H).half(), (0.1 * randn(g, 1, H, E)).half()
    w1, b1, w2 = weight(g, E, H, F, torch.float16, "nk"), 0.3 * randn(g, E, F), weight(g, E, F, H, torch.float16, "kn")
    ids, tw = lib.route_logits(lib.linear(x, Wg, ws, out_dtype=torch.float32), k, renormalize=True)
    _, offsets, _, inv_pos, rows = lib.permute(d, ids, lib.workspace(d), x=x, want_x_perm=True)
    y = lib.linear(lib.linear(rows, w1, ws, bias=b1, activation="gelu", offsets=offsets), w2, ws, offsets=offsets)
    out = lib.combine_rows(y, inv_pos, tw, residual=x)
    assert out.dtype == torch.float16 and lib.check(ws) == lib.MOE_OK
    want = x.double()
    for j in range(k):
        e = ids[:, j].long()
        hid = act64("gelu", torch.einsum("th,thf->tf", x.double(), w1.double()[e]) + b1.double()[e])
        want = want + tw[:, j, None].double() * torch.einsum("tf,tfh->th", hid, w2.double()[e])
    # h and y are rounded to fp16 on the way, and the output: three half steps
    rel = float((out.double() - want).norm() / want.norm())
    assert rel <= 2.0 ** -11 * 3 ** 0.5, rel


# ------------------------------------------- linear behind a long kernel --

def test_hold_limits(lib):
    for ms in (0, -1, 6001):
        assert lib.load().moe_selftest_hold(ms, None) == 1


@gpu
@pytest.mark.parametrize("R", [5, 3000])
def test_linear_behind_a_long_kernel(lib, R):
    """A dense product is resident while the kernel before it still runs, here for longer
    than a wait's limit of 4 s: that is no time of its own waits."""
    g = gen(R)
    K, N = 1024, 2048
    a, w = randn(g, R, K).bfloat16(), weight(g, 1, K, N, torch.bfloat16, "kn")
    own = lib.linear_workspace()
    want = lib.linear(a, w, own)
    out = torch.zeros_like(want)
    lib.selftest_hold(4500)
    lib.linear(a, w, own, out=out)
    assert lib.check(own) == lib.MOE_OK
    assert torch.equal(out, want)


# ---------------------------------------------- linear: activations' values --

@gpu
def test_linear_gelu_of_each_value(lib, ws):
    """gelu point by point (through the bias, the sums being zero), relative to its value
    also where that is small. In steps of fp32: the fit of erfc 0.9; t = 1 / (1 + 0.305 |x|)
    2.5, 2.6 times that in the result; its polynomial 3; e^x 2 for ex2 and 1 for its
    argument; the products 1.5: below 16. Under the smallest normal number it may be 0."""
    N = 1 << 16
    a = torch.zeros(1, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(1, 64, N, dtype=torch.bfloat16, device="cuda")
    for lo, hi in ((-14.0, 9.0), (-4.0, 0.0), (-1e-3, 1e-3), (-9.0, -4.0)):
        x = torch.linspace(lo, hi, N, device="cuda")[None]
        got = lib.linear(a, w, ws, bias=x, activation="gelu", out_dtype=torch.float32)[0].double()
        want = act64("gelu", x[0].double())
        off = (got - want).abs() - 14 * 2.0 ** -126
        assert bool((off <= 16 * 2.0 ** -23 * want.abs()).all()), float((off / want.abs()).max()) * 2 ** 23
        # 16 bits: the fit 4.0e-6, the rest of it as above and the exponent's rounding, x^2 / 2 2.5 half
        # steps: below 2^-15, and the output's own half step
        for dt in (torch.bfloat16, torch.float16):
            got = lib.linear(a.to(dt), w.to(dt), ws, bias=x, activation="gelu")[0].double()
            least = 14 * 2.0 ** -126 if dt == torch.bfloat16 else 2.0 ** -25
            tol = torch.finfo(dt).eps / 2 * (1 + 2.0 ** -15) + 2.0 ** -15
            assert bool(((got - want).abs() <= tol * want.abs() + least).all())
    x = torch.tensor([[math.inf, -math.inf, math.nan, 0.0, -0.0, 3e38, -3e38, 1e-40]], device="cuda")
    for dt in (torch.float32, torch.bfloat16):
        got = lib.linear(a, w[:, :, :8].contiguous(), ws, bias=x, activation="gelu", out_dtype=dt)[0]
        assert got[0] == math.inf and got[1] == 0 and got[2].isnan() and bool((got[3:5] == 0).all())
        assert got[5] == x[0, 5].to(dt) and got[6] == 0 and abs(float(got[7])) <= 1e-40


@gpu
@pytest.mark.parametrize("act,lo", [("silu", -80.0), ("gelu_tanh", -9.0)])
def test_linear_silu_and_gelu_tanh_of_each_value(lib, ws, act, lo):
    """Their exponential e^-u is within 2.5 steps + 1.2 for each |u| of itself, u 1.5 steps, the sum
    and the quotient 2.5: 5 + 3 |u| together."""
    N = 1 << 16
    a = torch.zeros(1, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(1, 64, N, dtype=torch.bfloat16, device="cuda")
    x = torch.linspace(lo, 10.0, N, device="cuda")[None]
    got = lib.linear(a, w, ws, bias=x, activation=act, out_dtype=torch.float32)[0].double()
    v = x[0].double()
    u = v if act == "silu" else 2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)
    want = act64(act, v)
    assert bool(((got - want).abs() <= (5 + 3 * u.abs()) * 2.0 ** -23 * want.abs()).all())


# ----------------------------------------------------- linear: its schedules --

FEW, ONE, PAIR, HALF = range(4)
SCHEDULES = [   # form, how its tiles are cut, parts of a cut tile at most, K, N, rows of each group
    (FEW, "even", 2, 1280, 7552, [1]), (FEW, "even", 3, 1064, 4976, [3]), (FEW, "even", 15, 8192, 1000, [16]),
    (FEW, "uneven", 2, 984, 20496, [1]), (FEW, "uneven", 2, 1512, 40320, [7]), (FEW, "uneven", 3, 3008, 9840, [1]),
    (FEW, "uneven", 3, 9592, 12096, [16]), (FEW, "uneven", 4, 7176, 6480, [2]),
    (ONE, "even", 2, 4144, 8, [8653]), (ONE, "even", 2, 2496, 3680, [1, 1]), (ONE, "even", 3, 3184, 8, [5179]),
    (ONE, "even", 3, 1480, 8, [1, 0, 1, 0, 1, 5, 72, 1]), (ONE, "even", 5, 4368, 8, [3442]),
    (ONE, "uneven", 2, 2504, 16, [19486]), (ONE, "uneven", 2, 1376, 9896, [0, 1, 1]), (ONE, "uneven", 2, 2944, 39488, [38]),
    (ONE, "uneven", 3, 4376, 8, [9867]), (ONE, "uneven", 2, 2040, 104, [22554]), (ONE, "uneven", 4, 7296, 8, [6822]),
    (ONE, "uneven", 4, 14664, 1640, [0, 0, 1, 1, 0, 1, 1, 0]),
    (PAIR, "even", 2, 10232, 6480, [130]), (PAIR, "even", 3, 7464, 5408, [147]), (PAIR, "even", 3, 12856, 1208, [1280]),
    (PAIR, "even", 3, 8848, 136, [154, 0, 3, 0, 0, 1, 400, 353, 0, 0, 1013, 0, 0, 570, 2129, 11]),
    (PAIR, "uneven", 2, 4440, 20048, [161]), (PAIR, "uneven", 2, 6048, 3624, [1299]), (PAIR, "uneven", 2, 4384, 7872, [1270]),
    (PAIR, "uneven", 2, 4720, 3888, [786, 1]), (PAIR, "uneven", 2, 5312, 2624, [1580, 1710]),
    (PAIR, "uneven", 3, 11568, 10464, [132]),
    (PAIR, "uneven", 3, 15768, 272, [1, 1, 1, 0, 1, 40, 1, 1, 1, 0, 9, 66, 2255, 0, 0, 1]),
    (HALF, "even", 2, 2408, 8, [3698]), (HALF, "even", 2, 1656, 5800, [0, 1]), (HALF, "even", 3, 2200, 776, [500]),
    (HALF, "even", 5, 6000, 264, [330]), (HALF, "uneven", 2, 1440, 19624, [20]), (HALF, "uneven", 2, 1592, 39016, [18]),
    (HALF, "uneven", 2, 1552, 3304, [1, 0, 2, 1, 1, 1, 0, 1]), (HALF, "uneven", 3, 5576, 144, [4891]),
    (HALF, "uneven", 3, 4688, 464, [910, 0, 1, 1, 121, 2, 1, 1, 0, 0, 0, 1, 1, 366, 0, 1]),
    (HALF, "uneven", 4, 8872, 136, [3395]), (HALF, "uneven", 4, 8848, 24, [0, 1, 1, 1, 2641, 8, 38, 1]),
]


def how_cut(s):
    if not s.segments:
        return "whole"
    left = s.tiles - s.whole
    return "even" if s.segments % left == 0 and s.segments // left == s.most_parts else "uneven"


def walk_schedule(s, K, form):
    """Every run of a schedule, block by block, as the kernel walks it: each cut tile's blocks are
    computed once, its parts lie where its join reads them, and all of it in the workspace."""
    k_blocks, left, ctas = -(-K // 64), s.tiles - s.whole, 2 if form >= PAIR else 1
    total, pieces = left * k_blocks, {}
    assert total * (s.segments + 1) < 2 ** 32 and s.segments <= s.units
    for unit in range(s.segments):
        pos, end = total * unit // s.segments, total * (unit + 1) // s.segments
        assert pos < end
        while pos < end:
            q, kb0 = divmod(pos, k_blocks)
            kb1 = min(k_blocks, kb0 + end - pos)
            pieces.setdefault(q, []).append((kb0, kb1, unit))
            pos += kb1 - kb0
    assert sorted(pieces) == list(range(left))
    slots = set()
    for q, found in pieces.items():
        assert [a for a, _, _ in found] == [0] + [b for _, b, _ in found[:-1]] and found[-1][1] == k_blocks
        if len(found) == 1:
            continue
        first = ((q * k_blocks + 1) * s.segments - 1) // total
        last = ((q + 1) * k_blocks * s.segments - 1) // total
        written = [2 * unit + (kb0 == 0) for kb0, _, unit in found]
        assert [u for _, _, u in found] == list(range(first, last + 1)) and len(found) <= s.most_parts
        assert written == [2 * first + 1] + [2 * (first + i) for i in range(1, len(found))]
        assert not slots & set(written)
        slots |= set(written)
    # 512 tickets, one for each tile and CTA; 81920 rows of parts, of which a join reads up to 63 past its own
    assert left * ctas <= 512 and s.part_rows % 32 == 0
    assert not slots or (max(slots) + 1) * s.part_rows * ctas + 63 <= 81920


def test_linear_schedules(lib):
    """What test_linear_of_every_schedule runs is what its list says; of each form whole tiles, even and
    uneven cuts and joins of two, three and more parts are there."""
    seen = set()
    for form, cut, parts, K, N, counts in SCHEDULES:
        s = lib.linear_schedule_selftest(counts, K, N)
        assert (s.form, how_cut(s), s.most_parts) == (form, cut, parts), (K, N, counts, s.form, how_cut(s), s.most_parts)
        walk_schedule(s, K, form)
        seen.add((form, cut, min(parts, 4), s.whole > 0))
        assert s.form == lib.linear_form_selftest(sum(counts), K, N, len(counts))
    assert {(f, c, p) for f, c, p, _ in seen} >= {(f, c, p) for f in range(4) for c in ("even", "uneven") for p in (2, 3)}
    assert {(f, p) for f, c, p, _ in seen if c == "uneven"} >= {(FEW, 4), (ONE, 4), (HALF, 4)}
    assert {f for f, c, _, rounds in seen if c == "uneven" and rounds} == {FEW, ONE, PAIR, HALF}
    assert lib.linear_schedule_selftest([0, 0], 64, 64).tiles == 0
    for bad in ([-1], [0, -1], [5, -1, 3]):
        with pytest.raises(lib.MoeError):
            lib.linear_schedule_selftest(bad, 64, 64)


def test_linear_schedules_fit_the_workspace(lib):
    rng = random.Random(7)

    def log_int(lo, hi, step=1):
        return max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step) * step)

    cuts = set()
    for _ in range(4000):
        G = rng.choice([1, 1, 2, 8, 64, 256])
        counts = [log_int(1, 100000) if G == 1 else rng.choice([0, 1, log_int(1, 4000)]) for _ in range(G)]
        K, N, sms = log_int(8, 60000, 8), log_int(8, 60000, 8), rng.choice([152, 152, 148, 76, 20, 2, 1])
        if not sum(counts):
            continue
        s = lib.linear_schedule_selftest(counts, K, N, sms)
        assert s.whole <= s.tiles and (s.segments > 0) == (s.whole < s.tiles)
        if s.segments:
            walk_schedule(s, K, s.form)
            cuts.add((s.form, how_cut(s), sms >= 148))
    assert len(cuts) >= 12


@gpu
@pytest.mark.parametrize("form,cut,parts,K,N,counts", SCHEDULES,
                         ids=lambda v: str(v) if not isinstance(v, list) else f"{len(v)}g{sum(v)}r")
@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_linear_of_every_schedule(lib, form, cut, parts, K, N, counts, layout):
    """Joins of cut tiles of every form: with the whole epilogue, twice with the same bits, the
    workspace's head left as found (no ticket, no error), rows of no group left alone."""
    g = gen(K + N + form)
    G, R = len(counts), sum(counts)
    a, w = randn(g, R, K).bfloat16(), weight(g, G, K, N, torch.bfloat16, layout)
    off, ends = offsets_of(counts)
    bias, res = randn(g, G, N), randn(g, R, N)
    ws = lib.linear_workspace()
    out = [torch.full((R + 2, N), -7.0, device="cuda") for _ in range(2)]
    for o in out:
        lib.linear(a, w, ws, bias=bias, activation="silu", residual=res, offsets=off, out_dtype=torch.float32, out=o[1:R + 1])
    assert not bool(ws[: lib.LINEAR_WORKSPACE_ZEROS].any())
    assert torch.equal(out[0], out[1]) and bool((out[0][[0, -1]] == -7.0).all())
    check_linear(out[0][1:-1], *linear64(a, w, ends, bias, "silu", res), K)
    # the early residual (no activation), in place
    both = torch.cat([res, res]).bfloat16()[:R]
    want = lib.linear(a, w, ws, bias=bias, residual=both, offsets=off)
    assert torch.equal(lib.linear(a, w, ws, bias=bias, residual=both, offsets=off, out=both), want)
    assert not bool(ws[: lib.LINEAR_WORKSPACE_ZEROS].any())


@gpu
@pytest.mark.parametrize("G,K,N", [(8, 4096, 256), (16, 2048, 1408), (4, 7168, 2048)])
def test_linear_of_skewed_groups(lib, ws, G, K, N):
    """The form goes by the rows' mean, the schedule by the rows that there are: nearly all rows in
    one group, in the first, the last, and none but one."""
    R = 1024
    for hot in (0, G // 2, G - 1):
        for rest in (0, 3):
            g = gen(hot + rest)
            counts = [rest] * G
            counts[hot] = R - rest * (G - 1)
            off, ends = offsets_of(counts)
            a, w = randn(g, R, K).bfloat16(), weight(g, G, K, N, torch.bfloat16, "kn")
            out = lib.linear(a, w, ws, offsets=off, out_dtype=torch.float32)
            assert lib.check(ws) == lib.MOE_OK
            check_linear(out, *linear64(a, w, ends), K)


# ------------------------------------------------------- linear: any number of columns --

def test_linear_columns_on_the_host(lib):
    """Weights with contiguous k may have any number of columns; those with contiguous n a
    multiple of 8. (No GPU here: what is accepted ends at the missing device.)"""
    need = lib.load().moe_linear_workspace_size()
    p, ws = ctypes.c_void_p(256), ctypes.c_void_p(4096)

    def call(layout, K, N):
        return lib.load().moe_linear(4, K, N, 1, 0, p, K, None, p, layout, None, 0, p, N, ws, need, None)

    assert call(0, 64, 60) == 2 and call(0, 64, 1) == 2 and call(1, 60, 64) == 2 and call(1, 64, 0) == 1
    if not torch.cuda.is_available():
        assert call(1, 64, 60) == call(1, 64, 1) == call(0, 64, 64) not in (0, 1, 2, 3)


@gpu
@pytest.mark.parametrize("N", [1, 4, 60, 65, 129, 255, 261])
@pytest.mark.parametrize("K,counts", [(2048, [3]), (264, [200]), (4096, [300]), (512, [6000]), (4160, [900]), (72, [5, 0, 130, 1]),
                                      (128, [700, 1, 900]), (14336, [2, 40])])
@pytest.mark.parametrize("out_dtype", ["bf16", "fp32"])
def test_linear_of_any_number_of_columns(lib, ws, N, K, counts, out_dtype):
    g = gen(N + K)
    R, G, od = sum(counts), len(counts), DTYPES[out_dtype]
    a, w = randn(g, R, K).bfloat16(), weight(g, G, K, N, torch.bfloat16, "nk")
    off, ends = offsets_of(counts)
    bias, res = randn(g, G, N), randn(g, R, N).to(od)
    wide = torch.full((R, N + 6), -7.0, dtype=od, device="cuda")
    out = lib.linear(a, w, ws, offsets=off, out_dtype=od, out=wide[:, 3:3 + N])
    assert lib.check(ws) == lib.MOE_OK
    assert bool((wide[:, :3] == -7).all()) and bool((wide[:, 3 + N:] == -7).all())
    check_linear(out, *linear64(a, w, ends), K)
    for act in (None, "gelu"):
        out = lib.linear(a, w, ws, bias=bias, activation=act, residual=res, offsets=off, out_dtype=od)
        check_linear(out, *linear64(a, w, ends, bias, act, res), K)
    if N % 8 and N > 1:
        with pytest.raises(lib.MoeError):
            lib.linear(a, w.contiguous(), ws, offsets=off)


@gpu
def test_route_from_the_logits_of_any_number_of_experts(lib, ws):
    g = gen(60)
    T, H, E, k = 333, 512, 60, 4
    x, Wg = randn(g, T, H).bfloat16(), randn(g, E, H).bfloat16() * 0.1
    logits = lib.linear(x, Wg[None].transpose(1, 2), ws, out_dtype=torch.float32)
    check_linear(logits, *linear64(x, Wg[None].transpose(1, 2), [0, T]), H)
    check_route(lib.route_logits(logits, k, renormalize=True), route64(logits, k, renormalize=True))


# ------------------------------------------------- route_logits: the weights' accuracy --

@gpu
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,spread", [(256, 8, 1, 1.0), (256, 8, 8, 12.0), (60, 4, 1, 30.0), (16, 8, 4, 4.0), (8, 2, 1, 3.0)])
@pytest.mark.parametrize("biased", [False, True])
def test_route_weights_accuracy(lib, scores, E, k, groups, spread, biased):
    """Half steps of fp32 (2^-24): a softmax score is e^d / the sum, d the distance to the largest
    logit: d's rounding |d|, e^d 6, the sum of 256 46, its reciprocal 2, a product and the scale 2;
    a sigmoid's e^-l 6, the sum 1, the reciprocal 2, the scale 1. Renormalized: twice a score's own
    (the sum over all experts cancels), 5 for the sum of 8, 4 for the quotient, the scale."""
    g = gen(E + k)
    x = spread * randn(g, 3000, E)
    bias = 0.05 * randn(g, E) if biased else None
    for renorm in (False, True):
        opts = dict(scores=scores, bias=bias, groups=groups, top_groups=max(1, groups // 2), renormalize=renorm, scale=2.5)
        ids, w = lib.route_logits(x, k, **opts)
        want_ids, want = route64(x, k, **opts)
        assert torch.equal(ids, want_ids)
        d = (x.amax(1, keepdim=True) - x.gather(1, ids.long())).double()
        steps = 56 + 2 * d if scores == "softmax" else 28.0
        off = ((w.double() - want).abs() - 2.5 * 2.0 ** -126) / want
        assert bool((off <= steps * 2.0 ** -24).all()), float((off / steps).max()) * 2 ** 24


@gpu
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [96, 160, 256])
@pytest.mark.parametrize("groups,top_groups,group_top", [(1, 1, 1), (8, 3, 1), (8, 3, 2)])
def test_route_forced_experts_of_many(lib, scores, E, groups, top_groups, group_top):
    """Infinite biases among several experts a lane, next to one another and in all groups; a
    bias of NaN puts its expert last."""
    g = gen(E)
    T, k = 4001, 8
    x = torch.randint(0, 4, (T, E), generator=g, device="cuda").float()
    for plus, minus, nan in (((5, 6, E - 1), (), ()), (range(0, E, 12), (3, 4), ()), (range(40), range(60, 80), (1, 90)), ((), (), (7,))):
        bias = torch.randint(0, 2, (E,), generator=g, device="cuda").float() * 2.0 ** -24
        for at, v in ((plus, math.inf), (minus, -math.inf), (nan, math.nan)):
            bias[list(at)] = v
        for renorm in (False, True):
            opts = dict(scores=scores, bias=bias, groups=groups, top_groups=top_groups, group_top=group_top, renormalize=renorm)
            idx = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
            w = torch.full((T, k), math.nan, device="cuda")
            lib.route_logits(x, k, topk_idx=idx, topk_w=w, **opts)
            check_route((idx, w), route64(x, k, **opts))
