"""Measured cases of the routing, product and combine operators: plain forms and the library's calls side by side.

Three operators that together are an expert layer whose router scores and whose experts are not
the fixed ones of the layer call (a balance bias, expert groups, experts with biases and another
activation), and that each stand next to the layer's own parts:

  route    route_logits  each token's k experts and weights from its logits: softmax or sigmoid
                         scores, a bias for balance in the selection, groups of experts of which
                         the best are kept, weights renormalized and scaled
  linear   linear        out = act(a W + bias) + residual for each group's (expert's) rows
  combine  combine_rows  out[t] = residual[t] + sum_j w[t, j] y[inv_pos[t, j]]: the experts' rows
                         back in token order

``run`` computes a case in its plain form (torch operations in 32 bits; the scores that decide
between experts in 64) or, where the module's ``own`` is set, through the library. ``exact`` is
each operator's definition in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one token of a decode step over 64 experts: launch latency
        {"name": "route-one-token", "op": "route", "T": 1, "E": 64, "k": 6, "dtype": "fp32", "scores": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "group_top": 1, "renorm": True, "scale": 1.0},
        # a ragged batch, an odd number of experts a group, the best groups by their best expert
        {"name": "route-ragged-groups", "op": "route", "T": 5003, "E": 160, "k": 6, "dtype": "bf16",
         "scores": "softmax", "bias": False, "groups": 8, "top_groups": 3, "group_top": 1, "renorm": False,
         "scale": 16.0},
        # a prefill over many experts with a balance bias: groups by the sum of their two best
        {"name": "route-prefill-bias", "op": "route", "T": 32768, "E": 256, "k": 8, "dtype": "fp32",
         "scores": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "group_top": 2, "renorm": True,
         "scale": 2.5},
        # one token through a wide dense projection with bias and activation: weight streaming
        {"name": "linear-one-token", "op": "linear", "T": 1, "k": 1, "E": 1, "K": 4096, "N": 14336, "dtype": "bf16",
         "out": "bf16", "layout": "kn", "act": "gelu", "bias": True, "residual": False},
        # a decode batch on many narrow experts, a handful of rows each
        {"name": "linear-decode-experts", "op": "linear", "T": 128, "k": 6, "E": 64, "K": 2048, "N": 1408,
         "dtype": "bf16", "out": "bf16", "layout": "kn", "act": "relu", "bias": True, "residual": False},
        # the router's logits of a prefill, in 32 bits
        {"name": "linear-logits-fp32", "op": "linear", "T": 8192, "k": 1, "E": 1, "K": 4096, "N": 256,
         "dtype": "bf16", "out": "fp32", "layout": "kn", "act": "none", "bias": False, "residual": False},
        # a ragged batch on 64 experts, about a hundred rows each, weights with contiguous K
        {"name": "linear-ragged-fp16", "op": "linear", "T": 789, "k": 8, "E": 64, "K": 3584, "N": 2560,
         "dtype": "fp16", "out": "fp16", "layout": "nk", "act": "silu", "bias": True, "residual": False},
        # a prefill's projection back into the residual stream
        {"name": "linear-residual", "op": "linear", "T": 8192, "k": 1, "E": 1, "K": 4096, "N": 4096, "dtype": "bf16",
         "out": "bf16", "layout": "nk", "act": "none", "bias": True, "residual": True},
        # a prefill on wide experts: bound by the tensor cores
        {"name": "linear-prefill-experts", "op": "linear", "T": 8192, "k": 2, "E": 8, "K": 4096, "N": 14336,
         "dtype": "bf16", "out": "bf16", "layout": "kn", "act": "gelu_tanh", "bias": True, "residual": False},
        # one token's experts back to its row: launch latency
        {"name": "combine-one-token", "op": "combine", "T": 1, "H": 4096, "k": 2, "dtype": "bf16", "out": "bf16",
         "residual": True, "dropped": False},
        # an odd number of tokens with the residual stream in 32 bits, assignments over capacity dropped
        {"name": "combine-dropped-fp32", "op": "combine", "T": 1531, "H": 3584, "k": 8, "dtype": "bf16", "out": "fp32",
         "residual": True, "dropped": True},
        # the longest prefill on many narrow experts
        {"name": "combine-prefill", "op": "combine", "T": 32768, "H": 2048, "k": 6, "dtype": "bf16", "out": "bf16",
         "residual": True, "dropped": False},
    ]


MOST_FLOPS = 1.9e12                 # of the listed cases' largest (2 R K N)
MOST_WEIGHTS = 8 * 4096 * 14336
MOST_ROWS = 32768 * 6 * 2048        # values that a combine reads


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def _draw_route(rng):
    E = rng.choice([8, 60, 64, 128, 160, 256, rng.randint(9, 256)])
    group_top = rng.choice([1, 2])
    groups = rng.choice([g for g in range(1, 33) if E % g == 0 and E // g >= group_top])
    if rng.random() < 0.4:
        groups = 1
    top_groups = rng.randint(1, groups)
    return {"op": "route", "T": _log_int(rng, 1, 32768), "E": E, "k": rng.randint(1, min(8, top_groups * E // groups)),
            "dtype": rng.choice(["fp32", "fp32", "bf16", "fp16"]), "scores": rng.choice(["softmax", "sigmoid"]),
            "bias": rng.random() < 0.5, "groups": groups, "top_groups": top_groups, "group_top": group_top,
            "renorm": rng.random() < 0.6, "scale": rng.choice([1.0, 2.5, 16.0])}


def _draw_linear(rng):
    E, k = rng.choice([(1, 1), (1, 1), (8, 2), (16, 4), (64, 6), (64, 8), (128, 8), (256, 8)])
    while True:
        K, N = _log_int(rng, 64, 14336, 8), _log_int(rng, 64, 14336, 8)
        if E * K * N <= MOST_WEIGHTS:
            break
    T = _log_int(rng, 1, max(1, min(32768, int(MOST_FLOPS / (2.0 * k * K * N)))))
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    return {"op": "linear", "T": T, "k": k, "E": E, "K": K, "N": N, "dtype": dtype,
            "out": rng.choice([dtype, dtype, "fp32"]), "layout": rng.choice(["kn", "nk"]),
            "act": rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]), "bias": rng.random() < 0.6,
            "residual": rng.random() < 0.4}


def _draw_combine(rng):
    H, k = rng.choice([2048, 3584, 4096, _log_int(rng, 64, 16384, 8)]), rng.randint(1, 8)
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    T = _log_int(rng, 1, min(32768, MOST_ROWS // (H * k * (2 if dtype == "fp32" else 1))))
    return {"op": "combine", "T": T, "H": H, "k": k, "dtype": dtype, "out": rng.choice([dtype, "fp32"]),
            "residual": rng.random() < 0.6, "dropped": rng.random() < 0.3}


def draw(rng: random.Random):
    return rng.choice([_draw_route, _draw_linear, _draw_combine])(rng)


def _size(dtype):
    return 4 if dtype == "fp32" else 2


def work(case):
    T, k = case["T"], case["k"]
    if case["op"] == "route":
        E = case["E"]
        # the logits (and bias) read, ids and weights written
        return {"bytes": T * E * _size(case["dtype"]) + 4 * E * case["bias"] + 8 * T * k, "flops": 0}
    if case["op"] == "combine":
        H, R = case["H"], T * k * (0.9 if case["dropped"] else 1.0)
        return {"bytes": int(R * H) * _size(case["dtype"]) + T * H * _size(case["out"]) * (1 + case["residual"]) + 8 * T * k,
                "flops": 2.0 * R * H}
    E, K, N = case["E"], case["K"], case["N"]
    R = T * k
    active = min(E, max(k, round(E * (1 - (1 - k / E) ** T))))   # experts that get a row
    return {"bytes": 2 * R * K + active * N * (2 * K + 4 * case["bias"]) + R * N * _size(case["out"]) * (1 + case["residual"]),
            "flops": 2.0 * R * K * N}


# ----------------------------------------------------------------- inputs --

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, R, K):
    """Rows with a few channels far larger than the others, as layers see them."""
    gain = torch.exp(0.5 * _randn(g, K))
    gain = torch.where(torch.rand(K, generator=g, device="cuda") < 0.01, 8 * gain, gain)
    return _randn(g, R, K) * gain


def _topk(g, T, E, k):
    """k distinct experts for each token."""
    return _randn(g, T, E).topk(k, -1).indices


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    state = {"case": case}
    T, k, dt = case["T"], case["k"], DTYPES[case["dtype"]]
    if case["op"] == "route":
        E = case["E"]
        state["logits"] = (1.5 * _randn(g, T, E) + 0.7 * _randn(g, E)).to(dt)
        spread = 0.1 if case["scores"] == "sigmoid" else 0.5 / E
        state["bias"] = spread * _randn(g, E) if case["bias"] else None
        return state
    out = DTYPES[case["out"]]
    if case["op"] == "combine":
        H, R = case["H"], T * k
        # where each assignment's row lies: the assignments sorted by expert
        order = torch.argsort(_topk(g, T, 64, k).flatten(), stable=True)
        inv = torch.empty(R, dtype=torch.int32, device="cuda")
        inv[order] = torch.arange(R, dtype=torch.int32, device="cuda")
        if case["dropped"]:
            inv[torch.rand(R, generator=g, device="cuda") < 0.1] = -1
        state["inv_pos"], state["w"] = inv, torch.softmax(_randn(g, T, k), -1)
        state["y"] = _randn(g, R, H).to(dt)
        state["residual"] = (2 * _activations(g, T, H)).to(out) if case["residual"] else None
        return state
    E, K, N = case["E"], case["K"], case["N"]
    counts = torch.bincount(_topk(g, T, E, k).flatten(), minlength=E)
    state["offsets"] = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).to(torch.int32) if E > 1 else None
    state["active"], state["most"] = counts.nonzero().flatten(), int(counts.max())
    state["a"] = _activations(g, T * k, K).to(dt)
    # [E, K, N], its memory with contiguous N or K
    w = torch.empty(E, K, N, dtype=dt, device="cuda")
    if case["layout"] == "nk":
        w = torch.empty(E, N, K, dtype=dt, device="cuda").transpose(1, 2)
    for e in range(E):
        w[e] = (K ** -0.5 * _randn(g, K, N)).to(dt)
    state["w"] = w
    state["bias"] = 0.1 * _randn(g, E, N) if case["bias"] else None
    state["residual"] = (2 * _activations(g, T * k, N)).to(out) if case["residual"] else None
    return state


# -------------------------------------------------------------------- run --

def _plain_route(s):
    case, k = s["case"], s["case"]["k"]
    logits = s["logits"].double()   # which of two near scores is larger wants more than 32 bits
    if case["scores"] == "softmax":
        e = torch.exp(logits - logits.amax(-1, keepdim=True))
        score = e / e.sum(-1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-logits))
    biased = score if s["bias"] is None else score + s["bias"].double()
    key = logits if s["bias"] is None else biased   # without a bias scores are in their logits' order
    if case["groups"] > 1:
        two = case["group_top"] == 2
        best = (biased if two else key).unflatten(-1, (case["groups"], -1)).sort(dim=-1, descending=True).values
        best = best[..., 0] + best[..., 1] if two else best[..., 0]
        place = best.sort(dim=-1, descending=True, stable=True).indices.argsort(-1)
        kept = (place < case["top_groups"]).repeat_interleave(case["E"] // case["groups"], -1)
        key = torch.where(kept, key, -math.inf)
    ids = key.sort(dim=-1, descending=True, stable=True).indices[:, :k]   # ties to the lowest index
    w = score.gather(-1, ids)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return {"ids": ids.to(torch.int32), "w": (w * case["scale"]).float()}


def _plain_act(name, v):
    if name == "relu":
        return torch.clamp(v, min=0)
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * 0.5 ** 0.5))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh((2 / math.pi) ** 0.5 * (v + 0.044715 * v * v * v)))
    return v


def _plain_linear(s):
    case, a, w = s["case"], s["a"], s["w"]
    if s["offsets"] is None:
        v = a.float() @ w[0].float()
        if s["bias"] is not None:
            v = v + s["bias"][0]
    else:
        # the experts that have rows, each one's rows padded to the longest, in one batched product
        rows = torch.arange(a.shape[0], device=a.device)
        expert = torch.searchsorted(s["offsets"][1:], rows, right=True)
        slot = torch.searchsorted(s["active"], expert) * s["most"] + rows - s["offsets"][expert]
        padded = torch.zeros(s["active"].shape[0] * s["most"], case["K"], device=a.device)
        padded[slot] = a.float()
        v = torch.bmm(padded.unflatten(0, (-1, s["most"])), w[s["active"]].float()).flatten(0, 1)[slot]
        if s["bias"] is not None:
            v = v + s["bias"][expert]
    v = _plain_act(case["act"], v)
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return {"out": v.to(DTYPES[case["out"]])}


def _plain_combine(s):
    case = s["case"]
    at = s["inv_pos"].view(case["T"], case["k"])
    w = torch.where(at >= 0, s["w"], 0.0)
    v = (s["y"].float()[at.clamp(min=0)] * w.unsqueeze(-1)).sum(1)
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return {"out": v.to(DTYPES[case["out"]])}


_kept = {}   # the workspace that a program keeps


def _run_own(s):
    from token_dispatch_grouped_moe_gb300 import lib
    case = s["case"]
    if case["op"] == "route":
        ids, w = lib.route_logits(s["logits"], case["k"], scores=case["scores"], bias=s["bias"], groups=case["groups"],
                                  top_groups=case["top_groups"], group_top=case["group_top"],
                                  renormalize=case["renorm"], scale=case["scale"])
        return {"ids": ids, "w": w}
    out = DTYPES[case["out"]]
    if case["op"] == "combine":
        return {"out": lib.combine_rows(s["y"], s["inv_pos"], s["w"], residual=s["residual"], out_dtype=out)}
    if "ws" not in _kept:
        _kept["ws"] = lib.linear_workspace()
    return {"out": lib.linear(s["a"], s["w"], _kept["ws"], bias=s["bias"],
                              activation=None if case["act"] == "none" else case["act"], residual=s["residual"],
                              offsets=s["offsets"], out_dtype=out)}


def run(state):
    if own:
        return _run_own(state)
    return {"route": _plain_route, "linear": _plain_linear, "combine": _plain_combine}[state["case"]["op"]](state)


# ------------------------------------------------------------------ exact --

def _places(v):
    """Each value's place in its row's descending order, equal ones by index: how many come before it."""
    n = v.shape[-1]
    index = torch.arange(n, device=v.device)
    lower = index[None, :] < index[:, None]
    x, y = v.unsqueeze(-1), v.unsqueeze(-2)
    return ((y > x) | ((y == x) & lower)).sum(-1)


def _exact_route(s, lo, hi):
    case = s["case"]
    E, k, groups = case["E"], case["k"], case["groups"]
    x = s["logits"][lo:hi].double()
    if case["scores"] == "softmax":
        score = torch.softmax(x, 1)
    else:
        score = torch.sigmoid(x)
    choice = score if s["bias"] is None else score + s["bias"].double()
    order = x if s["bias"] is None else choice
    if groups > 1:
        members = (order if case["group_top"] == 1 else choice).reshape(hi - lo, groups, E // groups)
        value = members.topk(case["group_top"], 2).values.sum(2)
        allowed = (_places(value) < case["top_groups"])[:, torch.arange(E, device="cuda") // (E // groups)]
        order = order.masked_fill(~allowed, -math.inf)
    place = _places(order)
    ids = torch.stack([(place == j).int().argmax(1) for j in range(k)], 1)
    w = torch.stack([score[torch.arange(hi - lo, device="cuda"), ids[:, j]] for j in range(k)], 1)
    if case["renorm"]:
        w = w / sum(w[:, j] for j in range(k))[:, None]
    return ids.to(torch.int32), w * case["scale"]


def _exact_act(name, v):
    if name == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return v * 0.5 * torch.erfc(-v / math.sqrt(2))
    if name == "gelu_tanh":
        # 1 + tanh(u) = 2 / (1 + exp(-2u))
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        parts = [_exact_route(s, lo, min(lo + 1024, case["T"])) for lo in range(0, case["T"], 1024)]
        return {"ids": torch.cat([p[0] for p in parts]), "w": torch.cat([p[1] for p in parts])}
    if case["op"] == "combine":
        T, k = case["T"], case["k"]
        out = torch.zeros(T, case["H"], dtype=torch.float64, device="cuda")
        if s["residual"] is not None:
            out += s["residual"].double()
        at = s["inv_pos"].long().reshape(T, k)
        for j in range(k):
            there = (at[:, j] >= 0).nonzero().flatten()
            out[there] += s["w"][there, j, None].double() * s["y"][at[there, j]].double()
        return {"out": out}
    R, N = s["a"].shape[0], case["N"]
    out = torch.zeros(R, N, dtype=torch.float64, device="cuda")
    ends = [0, R] if s["offsets"] is None else s["offsets"].tolist()
    for e in range(case["E"]):
        lo, hi = ends[e], ends[e + 1]
        if hi > lo:
            v = s["a"][lo:hi].double() @ s["w"][e].double()
            if s["bias"] is not None:
                v = v + s["bias"][e].double()
            out[lo:hi] = _exact_act(case["act"], v)
    if s["residual"] is not None:
        out += s["residual"].double()
    return {"out": out}
