"""Measured cases of the 8-bit operators: plain forms and the library's calls side by side.

Three operators of an expert layer that is served with 8-bit floating-point (e4m3) weights
and activations, one 32-bit scale for each row's block of 128 activations and for each
128 x 128 block of a weight:

  norm    add_rmsnorm_fp8  r = x + residual, y = r / sqrt(mean(r^2) + eps) * weight, and y in
                           e4m3 with a scale for each row's block of 128
  gated   fp8_gated        h = silu(a W1^T) * (a W3^T) for each expert's rows, in e4m3 with scales
  matmul  fp8_matmul       out = a W^T for each expert's rows

``run`` computes a case in its plain form (torch operations in 32 bits) or, where the module's
``own`` is set, through the library. ``exact`` is each operator's definition in 64 bits.
"""
import math
import random

import torch

own = False

BLOCK = 128          # values that share one scale
E4M3_MAX = 448.0     # the largest e4m3 value
AMAX_MIN = 2.0 ** -100   # a block's largest magnitude counts as at least this
EPS = 1e-6
FP8 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token of the residual stream between two layers of a decode step: launch latency
        {"name": "norm-one-token", "op": "norm", "T": 1, "H": 4096, "dtype": "bf16", "residual": True},
        # a ragged batch with the residual stream kept in 32 bits
        {"name": "norm-ragged-fp32", "op": "norm", "T": 1531, "H": 3584, "dtype": "fp32", "residual": True},
        # a prefill of 8192 tokens at H = 4096
        {"name": "norm-prefill", "op": "norm", "T": 8192, "H": 4096, "dtype": "bf16", "residual": True},
        # the longest prefill, first layer of a stack: nothing to add
        {"name": "norm-long-first", "op": "norm", "T": 32768, "H": 2048, "dtype": "bf16", "residual": False},
        # one token through two of eight wide experts: weight streaming
        {"name": "gated-one-token", "op": "gated", "T": 1, "k": 2, "E": 8, "K": 4096, "N": 14336, "zipf": False},
        # a decode batch on many narrow experts: about a hundred rows for each
        {"name": "gated-batch", "op": "gated", "T": 1024, "k": 6, "E": 64, "K": 2048, "N": 1408, "zipf": False},
        # a prefill on many narrow experts: bound by the tensor cores
        {"name": "gated-prefill", "op": "gated", "T": 32768, "k": 6, "E": 64, "K": 2048, "N": 1408, "zipf": False},
        # the second product for one token on narrow experts: latency
        {"name": "matmul-one-token", "op": "matmul", "T": 1, "k": 6, "E": 64, "K": 1408, "N": 2048,
         "out": "bf16", "zipf": False},
        # an odd number of rows through one dense (shared) expert, 32-bit result for a later sum
        {"name": "matmul-dense-odd", "op": "matmul", "T": 333, "k": 1, "E": 1, "K": 20480, "N": 3584,
         "out": "fp32", "zipf": False},
        # a ragged batch on 64 experts
        {"name": "matmul-ragged", "op": "matmul", "T": 789, "k": 8, "E": 64, "K": 2560, "N": 3584,
         "out": "bf16", "zipf": False},
        # a prefill of wide experts under skewed routing
        {"name": "matmul-prefill-skewed", "op": "matmul", "T": 8192, "k": 2, "E": 8, "K": 14336, "N": 4096,
         "out": "bf16", "zipf": True},
    ]


MOST_FLOPS = 1.9e12         # of the listed cases' largest (2 R K N of the second product)
MOST_WEIGHTS = 8 * 14336 * 4096


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng: random.Random):
    op = rng.choice(["norm", "gated", "matmul"])
    if op == "norm":
        H = rng.choice([2048, 3584, 4096, _log_int(rng, 64, 16384, 16)])
        return {"op": op, "T": _log_int(rng, 1, min(32768, 8192 * 4096 // H)), "H": H,
                "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "residual": rng.random() < 0.75}
    E, k = rng.choice([(1, 1), (8, 2), (16, 4), (64, 6), (64, 8), (128, 8), (256, 8)])
    most = MOST_WEIGHTS // (2 if op == "gated" else 1)
    while True:
        K, N = _log_int(rng, 128, 14336, 16), _log_int(rng, 128, 14336, 16)
        if E * K * N <= most:
            break
    flops_per_token = 2.0 * k * K * N * (2 if op == "gated" else 1)
    T = _log_int(rng, 1, max(1, min(32768, int(MOST_FLOPS / flops_per_token))))
    case = {"op": op, "T": T, "k": k, "E": E, "K": K, "N": N, "zipf": E == 8 and rng.random() < 0.5}
    if op == "matmul":
        case["out"] = rng.choice(["bf16", "bf16", "fp32"])
    return case


def work(case):
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        size = 4 if case["dtype"] == "fp32" else 2
        # x, (residual, the sum written) and y, e4m3 and scales written, the weight read
        return {"bytes": T * H * (size * (4 if case["residual"] else 2) + 1) + 4 * T * -(-H // BLOCK) + size * H,
                "flops": 0}
    T, k, E, K, N = (case[n] for n in ("T", "k", "E", "K", "N"))
    R, kb, nb = T * k, -(-K // BLOCK), -(-N // BLOCK)
    active = min(E, max(k, round(E * (1 - (1 - k / E) ** T))))   # experts that get a row
    two = 2 if case["op"] == "gated" else 1
    out = R * (N + 4 * nb) if case["op"] == "gated" else R * N * (4 if case["out"] == "fp32" else 2)
    return {"bytes": R * (K + 4 * kb) + two * active * (N * K + 4 * nb * kb) + out,
            "flops": 2.0 * two * R * K * N}


# ----------------------------------------------------------------- inputs --

def _blocks(v, width=BLOCK):
    """v[..., n] as [..., ceil(n / width), width], zeros past the end."""
    pad = -v.shape[-1] % width
    if pad:
        v = torch.nn.functional.pad(v, (0, pad))
    return v.unflatten(-1, (-1, width))


def _quantize(y):
    """y (32 bits) in e4m3 with a scale for each row's block of 128."""
    blocks = _blocks(y)
    scale = blocks.abs().amax(-1).clamp(min=AMAX_MIN) / E4M3_MAX
    q = (blocks / scale.unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).flatten(-2)[..., : y.shape[-1]]
    return q.to(FP8).contiguous(), scale


def _activations(g, R, K):
    """Rows with a few channels far larger than the others, as layers see them."""
    gain = torch.exp(0.5 * torch.randn(K, generator=g, device="cuda"))
    gain = torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 8 * gain, gain)
    return torch.randn(R, K, generator=g, device="cuda") * gain


def _weights(g, E, N, K):
    """[E, N, K] e4m3 and the scales of its 128 x 128 blocks, about normal with deviation 0.02."""
    q = torch.empty(E, N, K, dtype=FP8, device="cuda")
    for e in range(E):
        q[e] = (torch.randn(N, K, generator=g, device="cuda") * 100).clamp(-E4M3_MAX, E4M3_MAX).to(FP8)
    scale = 0.0002 * (1 + 0.3 * torch.rand(E, -(-N // BLOCK), -(-K // BLOCK), generator=g, device="cuda"))
    return q, scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    state = {"case": case}
    if case["op"] == "norm":
        T, H, dt = case["T"], case["H"], DTYPES[case["dtype"]]
        state["x"] = torch.randn(T, H, generator=g, device="cuda").to(dt)
        state["residual"] = (2 * _activations(g, T, H)).to(dt) if case["residual"] else None
        state["weight"] = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(dt)
        return state
    T, k, E, K, N = (case[n] for n in ("T", "k", "E", "K", "N"))
    # rows in dispatch order: each token's k distinct experts, counted
    logits = torch.randn(T, E, generator=g, device="cuda")
    if case["zipf"]:
        logits = logits - 1.2 * torch.log(torch.arange(1, E + 1, device="cuda"))
    counts = torch.bincount(logits.topk(k, -1).indices.flatten(), minlength=E)
    state["offsets"] = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32)
    state["active"] = counts.nonzero().flatten()
    state["most"] = int(counts.max())
    state["a"], state["a_scale"] = _quantize(_activations(g, T * k, K))
    if case["op"] == "gated":
        state["w1"], state["w1_scale"] = _weights(g, E, N, K)
        state["w3"], state["w3_scale"] = _weights(g, E, N, K)
    else:
        state["w"], state["w_scale"] = _weights(g, E, N, K)
    return state


# -------------------------------------------------------------------- run --

def _spread(v, n):
    """One value for each block of 128 as one for each of n."""
    return v.repeat_interleave(BLOCK, -1)[..., :n]


def _grouped(s, w, w_scale):
    """Each expert's rows times its weight transposed, in 32 bits: the experts that have rows,
    each one's rows padded to the longest, in one batched product."""
    a, K, N = s["a"], w.shape[2], w.shape[1]
    rows = torch.arange(a.shape[0], device=a.device)
    expert = torch.searchsorted(s["offsets"][1:], rows, right=True)
    slot = torch.searchsorted(s["active"], expert) * s["most"] + rows - s["offsets"][expert]
    padded = torch.zeros(s["active"].shape[0] * s["most"], K, device=a.device)
    padded[slot] = a.float() * _spread(s["a_scale"], K)
    scale = _spread(_spread(w_scale[s["active"]], K).transpose(1, 2), N).transpose(1, 2)
    wf = w.view(torch.uint8)[s["active"]].view(FP8).float() * scale
    return torch.bmm(padded.unflatten(0, (-1, s["most"])), wf.transpose(1, 2)).flatten(0, 1)[slot]


def _run_plain(s):
    case = s["case"]
    if case["op"] == "norm":
        r = s["x"].float()
        if s["residual"] is not None:
            r = r + s["residual"].float()
        y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
        q, scale = _quantize(y)
        out = {"y": y.to(s["x"].dtype), "q": q, "scale": scale}
        if s["residual"] is not None:
            out["residual"] = r.to(s["x"].dtype)
        return out
    if case["op"] == "gated":
        gate = _grouped(s, s["w1"], s["w1_scale"])
        h, scale = _quantize(gate / (1 + torch.exp(-gate)) * _grouped(s, s["w3"], s["w3_scale"]))
        return {"h": h, "scale": scale}
    return {"out": _grouped(s, s["w"], s["w_scale"]).to(DTYPES[case["out"]])}


_kept = {}   # the workspace that a program keeps


def _run_own(s):
    from token_dispatch_grouped_moe_gb300 import lib
    case = s["case"]
    if case["op"] == "norm":
        r, y, q, scale = lib.add_rmsnorm_fp8(s["x"], s["weight"], residual=s["residual"], eps=EPS)
        out = {"y": y, "q": q, "scale": scale}
        if s["residual"] is not None:
            out["residual"] = r
        return out
    if "ws" not in _kept:
        _kept["ws"] = lib.fp8_workspace()
    if case["op"] == "gated":
        h, scale = lib.fp8_gated(s["a"], s["a_scale"], s["w1"], s["w1_scale"], s["w3"], s["w3_scale"], _kept["ws"],
                                 offsets=s["offsets"])
        return {"h": h, "scale": scale}
    return {"out": lib.fp8_matmul(s["a"], s["a_scale"], s["w"], s["w_scale"], _kept["ws"], offsets=s["offsets"],
                                  out_dtype=DTYPES[case["out"]])}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ exact --

def _e4m3_nearest(v):
    """v (64 bits, at most 448) rounded to the nearest e4m3 value, ties to even."""
    _, e = torch.frexp(v)                       # |v| = m 2^e, 1/2 <= m < 1
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_quantized(y):
    q, scales = torch.empty_like(y), []
    for c in range(0, y.shape[1], BLOCK):
        part = y[:, c: c + BLOCK]
        scale = torch.clamp(part.abs().max(1).values, min=AMAX_MIN) / E4M3_MAX
        q[:, c: c + BLOCK] = _e4m3_nearest(part / scale[:, None])
        scales.append(scale)
    return q, torch.stack(scales, 1)


def _exact_product(s, w, w_scale):
    R, K, N = s["a"].shape[0], w.shape[2], w.shape[1]
    col = torch.arange(K, device="cuda") // BLOCK
    row = torch.arange(N, device="cuda") // BLOCK
    out = torch.zeros(R, N, dtype=torch.float64, device="cuda")
    ends = s["offsets"].tolist()
    for e in s["active"].tolist():
        lo, hi = ends[e], ends[e + 1]
        a = s["a"][lo:hi].double() * s["a_scale"][lo:hi].double()[:, col]
        out[lo:hi] = a @ (w[e].double() * w_scale[e].double()[row][:, col]).T
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        r = s["x"].double()
        if case["residual"]:
            r = r + s["residual"].double()
        y = r / torch.sqrt((r * r).sum(1, keepdim=True) / case["H"] + EPS) * s["weight"].double()
        q, scale = _exact_quantized(y)
        out = {"y": y, "q": q, "scale": scale}
        if case["residual"]:
            out["residual"] = r
        return out
    if case["op"] == "gated":
        gate = _exact_product(s, s["w1"], s["w1_scale"])
        h, scale = _exact_quantized(gate * torch.sigmoid(gate) * _exact_product(s, s["w3"], s["w3_scale"]))
        return {"h": h, "scale": scale}
    return {"out": _exact_product(s, s["w"], s["w_scale"])}
