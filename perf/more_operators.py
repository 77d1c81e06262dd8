"""The operators of a feed-forward of ternary experts, as cases that can be timed.

Four operators, in the order a layer runs them:

* ``route``: each token's largest router logits choose its experts and their weights;
  (token, choice) pairs are sorted by expert, so that each expert's rows lie together.
* ``experts``: the pairs' int8 rows times their expert's packed ternary matrix, ragged
  by expert: gate and up with the activation between them, or one matrix alone.
* ``linear``: the same product with one matrix for all rows, as a dense layer runs it:
  bias, activation, gating and residual behind the product.
* ``combine``: each token's expert outputs, weighted, summed and joined with a residual.

With ``own`` false ``run`` computes them with elementary torch operations, with
``own`` true by the library's calls.  ``exact`` computes them in 64 bits.
"""

import functools
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda:0"

# (hidden, width of an expert, experts, chosen ones).  Hidden 2560 / 6912 and 4096 / 14336 are
# the feed-forward sizes this repository knows; "fine" cuts the former's into sixths.
MODELS = {"2b": (2560, 6912, 8, 2), "8b": (4096, 14336, 8, 2), "fine": (2560, 1152, 64, 6)}


def _route(name, tokens, experts, topk, dtype, score, masked=0.0, padded=0.0):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "topk": topk, "dtype": dtype,
            "score": score, "masked": masked, "padded": padded}


def _experts(name, tokens, k, n, experts, topk, act, gated, slots, bias, dtype, skew=0.0, padded=0.0, layout=1):
    return {"name": name, "op": "experts", "tokens": tokens, "k": k, "n": n, "experts": experts, "topk": topk,
            "act": act, "gated": gated, "slots": slots, "bias": bias, "dtype": dtype, "skew": skew,
            "padded": padded, "layout": layout}


def _linear(name, tokens, k, n, act, gated, bias, residual, dtype):
    return {"name": name, "op": "linear", "tokens": tokens, "k": k, "n": n, "act": act, "gated": gated,
            "bias": bias, "residual": residual, "dtype": dtype}


def _combine(name, tokens, k, experts, topk, y_dtype, dtype, residual, padded=0.0, layout=1):
    return {"name": name, "op": "combine", "tokens": tokens, "k": k, "experts": experts, "topk": topk,
            "y_dtype": y_dtype, "dtype": dtype, "residual": residual, "padded": padded, "layout": layout}


def _gate_up(name, model, tokens, act, dtype, **kw):
    hidden, width, experts, topk = MODELS[model]
    return _experts(name, tokens, hidden, width, experts, topk, act, True, False, False, dtype, **kw)


def _down(name, model, tokens, dtype, bias=False, **kw):
    hidden, width, experts, topk = MODELS[model]
    return _experts(name, tokens, width, hidden, experts, topk, "none", False, True, bias, dtype, **kw)


def listed():
    return [
        # one user's next token: launch latency alone
        _route("route 1 token", 1, 8, 2, "f32", "chosen"),
        # a serving step of 64 users over many small experts
        _route("route 64 users", 64, 64, 6, "bf16", "softmax"),
        # prompts together, the batch padded at its end, a few experts switched off
        _route("route prompts", 16384, 256, 8, "f32", "sigmoid", masked=0.02, padded=0.05),
        # one user's next token: two experts' gate and up
        _gate_up("experts 1 token", "2b", 1, "relu2", "bf16"),
        # a serving step of 64 users: every expert gets a few rows
        _gate_up("experts 64 users", "fine", 64, "silu", "bf16"),
        # a long prompt
        _gate_up("experts prompt", "2b", 4096, "relu2", "bf16"),
        # parts of prompts, some experts far busier than others, a padded batch, fp32 between layers
        _down("experts uneven", "fine", 1003, "f32", bias=True, skew=1.0, padded=0.1),
        # a prompt through the widest experts' down projection
        _down("experts down", "8b", 2048, "bf16"),
        # one user's next token: the projection behind attention joins the residual stream
        _linear("linear 1 token", 1, 2560, 2560, "none", False, False, True, "bf16"),
        # a prompt through an up projection with bias and activation
        _linear("linear prompt", 2048, 4096, 14336, "gelu", False, True, False, "bf16"),
        # one user's next token
        _combine("combine 1 token", 1, 2560, 8, 2, "bf16", "bf16", True),
        # parts of prompts over small experts, fp32 residual stream, a padded batch
        _combine("combine prompts", 4093, 2560, 64, 6, "bf16", "f32", True, padded=0.1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["route", "experts", "experts", "linear", "combine"])
        dtype = rng.choice(["bf16", "f32"])
        act = rng.choice(["none", "relu2", "silu", "gelu"])
        gated, bias = rng.random() < 0.5, rng.random() < 0.3
        experts = rng.choice([8, 64, _log_int(rng, 1, 128)])
        topk = rng.randint(1, min(8, experts))
        padded, layout = rng.choice([0.0, 0.0, rng.uniform(0.0, 0.5)]), rng.randrange(1 << 20)
        k = rng.choice([2560, 4096, 64 * _log_int(rng, 1, 224)])
        n = rng.choice([2560, 6912, _log_int(rng, 1, 14336)])
        if op == "route":
            experts = rng.choice([experts, _log_int(rng, 2, 512)])
            case = _route("", _log_int(rng, 1, 16384), experts, min(topk, experts), dtype,
                          rng.choice(["softmax", "chosen", "sigmoid"]), rng.choice([0.0, 0.1, 0.9]), padded)
        elif op == "experts":
            case = _experts("", _log_int(rng, 1, 8192), k, n, experts, topk, act, gated, rng.random() < 0.5, bias,
                            dtype, skew=rng.choice([0.0, 0.5, 2.0]), padded=padded, layout=layout)
        elif op == "linear":
            case = _linear("", _log_int(rng, 1, 8192), k, n, act, gated, bias, rng.random() < 0.5, dtype)
        else:
            case = _combine("", _log_int(rng, 1, 8192), _log_int(rng, 1, 8192), experts, topk, dtype,
                            rng.choice(["bf16", "f32"]), rng.random() < 0.5, padded, layout)
        del case["name"]
        if _cost(case) <= most and _values(case) < 1e9:
            return case


def _values(case):
    """Weights, or values of the largest other array, that the case has."""
    if case["op"] == "route":
        return case["tokens"] * case["experts"]
    if case["op"] == "combine":
        return case["tokens"] * case["topk"] * case["k"]
    pairs = case["tokens"] * case.get("topk", 1)
    return max(case.get("experts", 1) * case["n"] * case["k"] * (1 + case["gated"]), pairs * max(case["k"], case["n"]))


@functools.lru_cache(maxsize=16)
def _chosen(tokens, experts, topk, skew, padded, layout):
    """[tokens, topk] distinct experts of each token; -1 for the padded tokens at the end."""
    g = np.random.default_rng(layout)
    liked = -skew * np.log1p(np.arange(experts))
    key = -(liked + g.gumbel(size=(tokens, experts)))
    out = np.argsort(key, axis=1, kind="stable")[:, :topk].astype(np.int32)
    out[tokens - int(padded * tokens):] = -1
    return out


def _choice(case):
    return _chosen(case["tokens"], case["experts"], case["topk"], case.get("skew", 0.0), case["padded"], case["layout"])


def _counts(case):
    """Rows of each expert."""
    e = _choice(case)
    return np.bincount(e[e >= 0], minlength=case["experts"]).tolist()


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _bytes(name):
    return 2 if name == "bf16" else 4


def work(case):
    if case["op"] == "route":
        m, e, k = case["tokens"], case["experts"], case["topk"]
        return {"bytes": m * e * _bytes(case["dtype"]) + 16 * m * k + 4 * (e + 1), "flops": 4 * m * e}
    es = _bytes(case["dtype"])
    if case["op"] == "combine":
        rows, m, k = sum(_counts(case)), case["tokens"], case["k"]
        return {"bytes": rows * k * _bytes(case["y_dtype"]) + m * k * es * (1 + case["residual"]) + 8 * m * case["topk"],
                "flops": 2 * rows * k}
    k, n, mats = case["k"], case["n"], 1 + case["gated"]
    if case["op"] == "experts":
        counts = _counts(case)
        rows, used = sum(counts), sum(c > 0 for c in counts)
        x_rows = rows if case["slots"] else int((_choice(case) >= 0).any(1).sum())
        more = 4 * rows + 4 * (case["experts"] + 1)
    else:
        rows, used, x_rows = case["tokens"], 1, case["tokens"]
        more = rows * n * es if case["residual"] else 0
    weights = used * mats * n * k // 4
    return {"bytes": weights + x_rows * (k + 4) + rows * n * es + more + used * mats * 4 * (1 + n * case["bias"]),
            "flops": 2 * rows * n * k * mats}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _packed(g, experts, n, k):
    """Ternary weights, 2 bits each, four a byte (codes q + 1, least significant pair first)."""
    trit = torch.arange(81, device=DEV)
    table = sum(((trit // 3 ** j) % 3) << (2 * j) for j in range(4)).to(torch.uint8)
    return table[torch.randint(0, 81, (experts, n, k // 4), generator=g, device=DEV)]


def _plan(expert, experts):
    """Slots sorted by expert, then by pair: first slot of each expert, pair of each slot, slot of each pair."""
    flat = expert.reshape(-1).long()
    pairs = flat.numel()
    key = torch.where(flat >= 0, flat, experts)
    order = torch.sort(key, stable=True).indices
    count = (key[:, None] == torch.arange(experts, device=DEV)).sum(0) if pairs * experts < 1 << 26 else \
        torch.zeros(experts + 1, dtype=torch.long, device=DEV).scatter_add_(0, key, torch.ones_like(key))[:experts]
    offset = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), count.cumsum(0)])
    used = torch.arange(pairs, device=DEV) < offset[-1]
    pair = torch.where(used, order, -1)
    slot = torch.empty_like(order)
    slot[order] = torch.where(used, torch.arange(pairs, device=DEV), -1)
    return offset.to(torch.int32), pair.to(torch.int32), slot.to(torch.int32).reshape(expert.shape)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device=DEV) * scale

    s = {"case": case}
    op, m = case["op"], case["tokens"]
    if op == "route":
        # logits of a trained router: a few experts stand out, some are liked by all tokens
        e = case["experts"]
        x = normal(m, e, scale=1.5) + normal(e, scale=0.5)
        off = torch.rand(e, generator=g, device=DEV) < case["masked"]
        x = torch.where(off, torch.full_like(x, -math.inf), x)
        x[m - int(case["padded"] * m):] = -math.inf
        s["logits"] = x.to(_dtype(case["dtype"])).contiguous()
        s["scale"] = 2.5 if case["score"] == "sigmoid" else 1.0
        if own:
            from ternary_weight_linear_bit_amd import _native as N
            s["routing"] = N.Routing.empty(m, case["topk"], e, device=DEV)
        return s
    dt = _dtype(case["dtype"])
    if op in ("experts", "combine"):
        s["expert"] = torch.from_numpy(_choice(case).copy()).to(DEV)
        s["offset"], s["pair"], s["slot"] = _plan(s["expert"], case["experts"])
        s["weight"] = torch.softmax(normal(m, case["topk"]), -1)
        s["counts"] = _counts(case)
    if op == "combine":
        k = case["k"]
        s["y"] = normal(m * case["topk"], k, scale=0.7).to(_dtype(case["y_dtype"]))
        s["residual"] = normal(m, k, scale=3.0).to(dt) if case["residual"] else None
        s["out"] = torch.empty(m, k, dtype=dt, device=DEV)
    else:
        n, k, mats, e = case["n"], case["k"], 1 + case["gated"], case.get("experts", 1)
        rows = m * case["topk"] if op == "experts" else m
        x_rows = rows if op == "linear" or case["slots"] else m
        s["x_q"] = normal(x_rows, k, scale=36.0).round_().clamp_(-127, 127).to(torch.int8)
        s["x_scale"] = normal(x_rows, scale=0.15).exp() * (3.6 / 127)
        s["w"] = [_packed(g, e, n, k) for _ in range(mats)]
        s["w_scale"] = [normal(e, scale=0.1).exp() * (2.0 / math.sqrt(k)) for _ in range(mats)]
        s["bias"] = [normal(e, n, scale=0.5) if case["bias"] else None for _ in range(mats)]
        s["residual"] = normal(m, n, scale=3.0).to(dt) if op == "linear" and case["residual"] else None
        # rows behind the last slot stay as they are
        s["out"] = torch.zeros(rows, n, dtype=dt, device=DEV)
    if own:
        from ternary_weight_linear_bit_amd import _native as N
        # the handles that a program keeps: a step's routing, weights in the matrix cores' layout
        if op != "linear":
            s["routing"] = N.Routing(s["expert"], s["weight"], s["offset"], s["pair"], s["slot"])
        if op == "experts":
            s["laid"] = [N.TernaryExperts.from_packed(w, c) for w, c in zip(s["w"], s["w_scale"])]
        elif op == "linear":
            s["laid"] = [(N.bitnet_repack_prefill(w[0]), c) for w, c in zip(s["w"], s["w_scale"])]
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if op == "route":
        return _run_route(s) if own else _plain_route(s)
    if op == "combine":
        return _run_combine(s) if own else _plain_combine(s)
    if op == "experts":
        return _run_experts(s) if own else _plain_experts(s)
    return _run_linear(s) if own else _plain_linear(s)


def _run_route(s):
    from ternary_weight_linear_bit_amd import _native as N
    r = N.bitnet_route(s["routing"], s["logits"], score=s["case"]["score"], scale=s["scale"])
    return {"expert": r.expert, "weight": r.weight, "offset": r.offset, "pair": r.pair, "slot": r.slot}


def _run_experts(s):
    from ternary_weight_linear_bit_amd import _native as N
    case, laid, bias = s["case"], s["laid"], s["bias"]
    gated = case["gated"]
    return N.bitnet_expert_linear(s["routing"], laid[0], s["x_q"], s["x_scale"], slots=case["slots"], act=case["act"],
                                  up=laid[1] if gated else None, bias=bias[0], up_bias=bias[1] if gated else None,
                                  y=s["out"])


def _run_linear(s):
    from ternary_weight_linear_bit_amd import _native as N
    case, laid, bias = s["case"], s["laid"], s["bias"]
    first = [None if b is None else b[0] for b in bias]
    gated = case["gated"]
    return N.bitnet_ternary_linear_act(*laid[0], case["n"], s["x_q"], s["x_scale"], act=case["act"],
                                       up=laid[1] if gated else None, bias=first[0],
                                       up_bias=first[1] if gated else None, residual=s["residual"], y=s["out"])


def _run_combine(s):
    from ternary_weight_linear_bit_amd import _native as N
    return N.bitnet_combine(s["routing"], s["y"], residual=s["residual"], out=s["out"])


def _plain_route(s):
    case = s["case"]
    m, topk = case["tokens"], case["topk"]
    x = s["logits"].float()
    at = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :topk]
    z = x.gather(1, at)
    some = z > -math.inf
    expert = torch.where(some, at, -1).to(torch.int32)
    if case["score"] == "sigmoid":
        w = 1 / (1 + (-z).exp())
    else:
        top = torch.where(some[:, :1], z[:, :1], torch.zeros_like(z[:, :1]))
        over = (z if case["score"] == "chosen" else x) - top
        total = over.exp().sum(1, keepdim=True)
        w = (z - top).exp() / torch.where(total > 0, total, torch.ones_like(total))
    weight = torch.where(some, w * s["scale"], torch.zeros_like(w))
    offset, pair, slot = _plan(expert, case["experts"])
    return {"expert": expert, "weight": weight, "offset": offset, "pair": pair, "slot": slot}


def _unpack(packed):
    """[N, K/4] bytes to the weights -1, 0, 1 as floats."""
    shift = torch.arange(0, 8, 2, device=DEV, dtype=torch.uint8)
    return (((packed[:, :, None] >> shift) & 3).float() - 1).reshape(packed.shape[0], -1)


def _activate(v, act):
    if act == "relu2":
        a = v.clamp(min=0)
        return a * a
    if act == "silu":
        return v / (1 + (-v).exp())
    if act == "gelu":
        return v * (0.5 * (1 + torch.erf(v * math.sqrt(0.5))))
    return v


def _plain_rows(s, e, x_q, x_scale):
    """The product, activation and gating of these rows with expert e's matrices."""
    x, v = x_q.float(), []
    for w, scale, bias in zip(s["w"], s["w_scale"], s["bias"]):
        acc = torch.matmul(x, _unpack(w[e]).T)
        v.append(acc * (scale[e] * x_scale)[:, None])
        if bias is not None:
            v[-1] = v[-1] + bias[e]
    a = _activate(v[0], s["case"]["act"])
    return a * v[1] if len(v) == 2 else a


def _plain_experts(s):
    case, at = s["case"], 0
    for e, count in enumerate(s["counts"]):
        if count:
            rows = torch.arange(at, at + count, device=DEV) if case["slots"] else \
                s["pair"][at:at + count].long() // case["topk"]
            s["out"][at:at + count] = _plain_rows(s, e, s["x_q"][rows], s["x_scale"][rows]).to(s["out"].dtype)
            at += count
    return s["out"]


def _plain_linear(s):
    a = _plain_rows(s, 0, s["x_q"], s["x_scale"])
    if s["residual"] is not None:
        a = a + s["residual"].float()
    s["out"].copy_(a)
    return s["out"]


def _plain_combine(s):
    out = torch.zeros(s["out"].shape, dtype=torch.float32, device=DEV)
    if s["residual"] is not None:
        out = s["residual"].float()
    for j in range(s["case"]["topk"]):
        at = s["slot"][:, j].long()
        y = s["y"][at.clamp(min=0)].float()
        out = out + torch.where(at[:, None] >= 0, s["weight"][:, j, None] * y, torch.zeros_like(y))
    s["out"].copy_(out)
    return s["out"]


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "experts": _exact_experts, "linear": _exact_linear, "combine": _exact_combine}[
        case["op"]](s)


def _exact_route(s):
    case = s["case"]
    m, e, topk = case["tokens"], case["experts"], case["topk"]
    x = s["logits"].double().cpu().numpy()
    number = np.broadcast_to(np.arange(e), (m, e))
    at = np.lexsort((number, -x))[:, :topk]                   # largest logit, then lowest number
    z = np.take_along_axis(x, at, 1)
    expert = np.where(np.isneginf(z), -1, at)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        if case["score"] == "sigmoid":
            w = 1 / (1 + np.exp(-z))
        else:
            over = z if case["score"] == "chosen" else x
            w = np.exp(z - np.logaddexp.reduce(over, axis=1)[:, None])
    weight = np.where(expert < 0, 0.0, w * s["scale"])
    lists = [[] for _ in range(e)]
    for p, c in enumerate(expert.reshape(-1).tolist()):
        if c >= 0:
            lists[c].append(p)
    offset = np.cumsum([0] + [len(v) for v in lists])
    pair, slot = np.full(m * topk, -1), np.full(m * topk, -1)
    pair[:offset[-1]] = [p for v in lists for p in v]
    slot[pair[:offset[-1]]] = np.arange(offset[-1])

    def whole(a):
        return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).to(DEV)
    return {"expert": whole(expert), "weight": torch.from_numpy(weight).to(DEV), "offset": whole(offset),
            "pair": whole(pair), "slot": whole(slot.reshape(m, topk))}


def _exact_product(s, i, e, x):
    """Rows x [rows, K] (64 bits, scaled) times matrix i of expert e, 2048 output rows at a time."""
    parts = []
    for w in s["w"][i][e].split(2048):
        q = torch.stack([(w // 4 ** j) % 4 for j in range(4)], -1).reshape(w.shape[0], -1).double() - 1
        parts.append(x @ q.T)
    v = torch.cat(parts, 1) * s["w_scale"][i][e].double()
    return v if s["bias"][i] is None else v + s["bias"][i][e].double()


def _exact_rows(s, e, x):
    v, act = _exact_product(s, 0, e, x), s["case"]["act"]
    if act == "relu2":
        v = torch.where(v > 0, v * v, torch.zeros_like(v))
    elif act == "silu":
        v = v * torch.sigmoid(v)
    elif act == "gelu":
        v = v * torch.special.ndtr(v)
    return v * _exact_product(s, 1, e, x) if s["case"]["gated"] else v


def _exact_experts(s):
    case = s["case"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    x = s["x_q"].double() * s["x_scale"].double()[:, None]
    flat = torch.from_numpy(_choice(case).reshape(-1).copy()).to(DEV)
    at = 0
    for e in range(case["experts"]):
        mine = torch.nonzero(flat == e)[:, 0]                 # pairs, ascending
        if len(mine):
            rows = torch.arange(at, at + len(mine), device=DEV) if case["slots"] else \
                torch.div(mine, case["topk"], rounding_mode="floor")
            out[at:at + len(mine)] = _exact_rows(s, e, x[rows])
            at += len(mine)
    return out


def _exact_linear(s):
    v = _exact_rows(s, 0, s["x_q"].double() * s["x_scale"].double()[:, None])
    return v if s["residual"] is None else v + s["residual"].double()


def _exact_combine(s):
    case = s["case"]
    flat = _choice(case).reshape(-1)
    order = np.argsort(np.where(flat < 0, case["experts"], flat), kind="stable")
    order = torch.from_numpy(order[:int((flat >= 0).sum())]).to(DEV)
    y = s["y"][:len(order)].double() * s["weight"].double().reshape(-1)[order][:, None]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV) if s["residual"] is None else \
        s["residual"].double()
    return out.index_add(0, torch.div(order, case["topk"], rounding_mode="floor"), y)
