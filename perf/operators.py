"""The operators between a layer's ternary products, as cases that can be timed.

Three operators of one decoder layer, in the order a layer runs them:

* ``append``: new keys and values are rotated by their position and written to a
  paged cache of 8-bit codes, one scale for each page and head; the queries are
  rotated on the way.
* ``attend``: attention of those queries over the cache, for single tokens, for
  a few drafted ones and for whole prompts.
* ``join``: the block's output, normalised, gated and scaled, joins the residual
  stream, and the next block's normalised input leaves as int8 codes.

With ``own`` false ``run`` computes them with elementary torch operations, with
``own`` true by the library's calls.  ``exact`` computes them in 64 bits.
"""

import math
import random

import torch

own = False

DEV = "cuda:0"
EPS = 1e-5

# Head counts (query, key/value) and widths of the layers this repository knows:
# hidden 2560 with 640 for k and v, hidden 4096 with 1024, hidden 8192 with 8192.
HEADS = {"2b": (20, 5, 128), "8b": (32, 8, 128), "100b": (64, 64, 128), "narrow": (12, 3, 64)}
WIDTHS = (2560, 4096, 6912, 8192, 14336)


def _append(name, shape, dtype, page, seqs, new, length, rot=128, pairs="halves", layout=1):
    return {"name": name, "op": "append", "shape": shape, "dtype": dtype, "page": page, "seqs": seqs,
            "new_lo": new[0], "new_hi": new[1], "len_lo": length[0], "len_hi": length[1], "rot": rot,
            "pairs": pairs, "layout": layout}


def _attend(name, shape, dtype, page, seqs, new, length, window=0, layout=1):
    return {"name": name, "op": "attend", "shape": shape, "dtype": dtype, "page": page, "seqs": seqs,
            "new_lo": new[0], "new_hi": new[1], "len_lo": length[0], "len_hi": length[1],
            "window": window, "layout": layout}


def _join(name, m, k, y_dtype, h_dtype, post, gate):
    return {"name": name, "op": "join", "m": m, "k": k, "y_dtype": y_dtype, "h_dtype": h_dtype,
            "post": post, "gate": gate}


def listed():
    return [
        # one user's next token in the 2B-shaped model: launch latency alone
        _append("append 1 token", "2b", "bf16", 64, 1, (1, 1), (1500, 1500)),
        # a serving step of the 8B-shaped model: 64 users at different lengths
        _append("append 64 users", "8b", "f32", 16, 64, (1, 1), (1, 8192)),
        # the prompt of one user of the 2B-shaped model
        _append("append prompt", "2b", "bf16", 64, 1, (4096, 4096), (4096, 4096)),
        # parts of seven prompts at once, behind what is cached; the widest model,
        # half of each head rotated, neighbouring dims paired
        _append("append 7 parts", "100b", "f32", 32, 7, (1, 501), (1, 3001), rot=64, pairs="neighbours"),
        # one user's next token in the 2B-shaped model
        _attend("attend 1 token", "2b", "bf16", 64, 1, (1, 1), (2049, 2049)),
        # a serving step of the 8B-shaped model: 64 users at different lengths
        _attend("attend 64 users", "8b", "bf16", 16, 64, (1, 1), (1, 8191)),
        # four long documents, next token, fp32 between layers
        _attend("attend long", "8b", "f32", 128, 4, (1, 1), (60001, 65536)),
        # drafted tokens checked in one pass, narrow heads, an odd number of users
        _attend("attend drafts", "narrow", "bf16", 32, 9, (1, 7), (5, 4099)),
        # a long prompt of the 8B-shaped model
        _attend("attend prompt", "8b", "bf16", 64, 1, (8192, 8192), (8192, 8192)),
        # parts of six prompts behind what is cached, the last 1024 tokens visible, fp32
        _attend("attend parts", "2b", "f32", 64, 6, (3, 701), (400, 4001), window=1024),
        # one user's next token in the 2B-shaped model
        _join("join 1 token", 1, 2560, "bf16", "bf16", True, "none"),
        # a prompt of the 8B-shaped model, a gate for each channel, fp32 residual stream
        _join("join prompt", 4093, 4096, "bf16", "f32", True, "channel"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["append", "attend", "attend", "join"])
        if op == "join":
            k = rng.choice([rng.choice(WIDTHS), _log_int(rng, 16, 16384)])
            case = _join("", _log_int(rng, 1, 8192), k, rng.choice(["bf16", "f32"]),
                         rng.choice(["bf16", "f32"]), rng.random() < 0.7,
                         rng.choice(["none", "channel", "token"]))
        else:
            shape = rng.choice(sorted(HEADS))
            page = rng.choice([16, 32, 64, 128])
            dtype = rng.choice(["bf16", "f32"])
            seqs = _log_int(rng, 1, 96)
            new_hi = rng.choice([1, 1, _log_int(rng, 2, 16), _log_int(rng, 16, 4096)])
            new_lo = 1 if rng.random() < 0.5 else new_hi
            len_hi = max(new_hi, _log_int(rng, 1, 32768))
            len_lo = rng.choice([1, len_hi, max(1, len_hi // 2)])
            if op == "append":
                case = _append("", shape, dtype, page, seqs, (new_lo, new_hi), (len_lo, len_hi),
                               rot=rng.choice([HEADS[shape][2], HEADS[shape][2] // 2]),
                               pairs=rng.choice(["halves", "neighbours"]), layout=rng.randrange(1 << 20))
            else:
                case = _attend("", shape, dtype, page, seqs, (new_lo, new_hi), (len_lo, len_hi),
                               window=rng.choice([0, 0, 0, _log_int(rng, 16, 8192)]),
                               layout=rng.randrange(1 << 20))
        del case["name"]
        if _cost(case) <= most and _plain_values(case) < 4e9:
            return case


def _plain_values(case):
    """Values of the largest array that the plain form makes of this case."""
    if case["op"] == "join":
        return case["m"] * case["k"]
    new, length, _, width = _lengths(case)
    hq, hk, dim = HEADS[case["shape"]]
    keys = width * case["page"]
    return case["seqs"] * keys * max(hk * dim, hq * max(new) if case["op"] == "attend" else 0)


def _lengths(case):
    """(new tokens, cached tokens with them) of each sequence, all new tokens, pages a row of the table."""
    rng = random.Random(case["layout"])
    new, length = [], []
    for _ in range(case["seqs"]):
        n = rng.randint(case["new_lo"], case["new_hi"])
        new.append(n)
        length.append(max(n, rng.randint(case["len_lo"], case["len_hi"])))
    return new, length, sum(new), -(-max(length) // case["page"])


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _bytes(name):
    return 2 if name == "bf16" else 4


def work(case):
    if case["op"] == "join":
        m, k = case["m"], case["k"]
        ey, eh = _bytes(case["y_dtype"]), _bytes(case["h_dtype"])
        gate = {"none": 0, "channel": k, "token": m * k}[case["gate"]] * ey
        norms = (8 if case["post"] else 4) * k
        return {"bytes": m * k * (ey + 2 * eh + 1) + gate + norms + 4 * m, "flops": 12 * m * k}
    new, length, tokens, _ = _lengths(case)
    hq, hk, dim = HEADS[case["shape"]]
    es, page = _bytes(case["dtype"]), case["page"]
    if case["op"] == "append":
        pages = sum((n + page - 1) // page for n in new)
        moved = tokens * dim * (2 * hk * (es + 1) + 2 * hq * es)
        return {"bytes": moved + 4 * tokens * case["rot"] + 8 * pages * hk + 4 * pages,
                "flops": tokens * (hq + hk) * case["rot"] * 3 + tokens * hk * dim * 6}
    pairs = keys = pages = 0
    window = case["window"]
    for n, ln in zip(new, length):
        first = ln - n                      # position of the first new token
        seen = min(ln, n + min(first, window - 1)) if window else ln
        keys += seen
        pages += -(-seen // page)
        if window:
            full = max(0, n - max(0, window - 1 - first))      # rows that see `window` keys
            low = n - full
            pairs += full * window + low * (first + 1) + low * (low - 1) // 2
        else:
            pairs += n * (first + 1) + n * (n - 1) // 2
    return {"bytes": 2 * keys * hk * dim + 8 * pages * hk + 4 * pages + 2 * tokens * hq * dim * es
            + 4 * tokens * hq, "flops": 4 * pairs * hq * dim}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _tables(positions, rot):
    """cos and sin of every position and pair of dims, made in 64 bits."""
    inv = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64, device=DEV) * 2 / rot)
    at = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * inv
    return at.cos().float().contiguous(), at.sin().float().contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device=DEV) * scale

    s = {"case": case}
    if case["op"] == "join":
        m, k = case["m"], case["k"]
        yd, hd = _dtype(case["y_dtype"]), _dtype(case["h_dtype"])
        s["y"] = normal(m, k, scale=0.7).to(yd)
        s["h"] = normal(m, k, scale=3.0).to(hd)
        s["h_out"] = torch.empty(m, k, dtype=hd, device=DEV)
        s["post"] = 1 + normal(k, scale=0.1) if case["post"] else None
        s["gate"] = {"none": lambda: None, "channel": lambda: (0.5 + normal(k, scale=0.2)).to(yd),
                     "token": lambda: normal(m, k).to(yd)}[case["gate"]]()
        s["pre"] = 1 + normal(k, scale=0.1)
        s["scale"] = 0.25
        return s
    new, length, tokens, width = _lengths(case)
    hq, hk, dim = HEADS[case["shape"]]
    page, seqs, dt = case["page"], case["seqs"], _dtype(case["dtype"])
    # pages in no order; every sequence its own
    counts = [-(-n // page) for n in length]
    order = torch.randperm(sum(counts) + 3, generator=g, device=DEV).to(torch.int32)
    at = torch.tensor([0] + counts, device=DEV).cumsum(0)
    col = torch.arange(width, device=DEV)
    index = (at[:-1, None] + col).clamp(max=sum(counts) - 1)
    s["table"] = torch.where(col < at.diff()[:, None], order[index], 0).to(torch.int32)
    pages = sum(counts) + 3
    s["q_start"] = torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32)
    s["kv_len"] = torch.tensor(length, dtype=torch.int32, device=DEV)
    s["max_new"], s["max_len"] = max(new), max(length)
    # what earlier tokens left: codes that use their page's range, scales near 4/127
    s["k"] = normal(pages, hk, page, dim, scale=36.0).round_().clamp_(-127, 127).to(torch.int8)
    s["v"] = normal(pages, hk, dim, page, scale=36.0).round_().clamp_(-127, 127).to(torch.int8)
    s["k_scale"] = (normal(pages, hk, scale=0.15).exp() * (3.6 / 127)).contiguous()
    s["v_scale"] = (normal(pages, hk, scale=0.15).exp() * (3.6 / 127)).contiguous()
    if case["op"] == "append":
        channel = 1 + 2 * (torch.rand(hk, dim, generator=g, device=DEV) < 0.02)
        s["new_k"] = (normal(tokens, hk, dim) * channel).to(dt)
        s["new_v"] = normal(tokens, hk, dim).to(dt)
        s["q"] = normal(tokens, hq, dim).to(dt)
        s["q_out"] = torch.empty_like(s["q"])
        s["cos"], s["sin"] = _tables(max(length), case["rot"])
    else:
        s["q"] = normal(tokens, hq, dim, scale=1.5).to(dt)
        s["out"] = torch.empty(tokens, hq, dim, dtype=dt, device=DEV)
        s["lse"] = torch.empty(tokens, hq, dtype=torch.float32, device=DEV)
        s["softmax_scale"] = dim ** -0.5
    if own:
        # the handles that a program keeps beside its cache and its batch
        from ternary_weight_linear_bit_amd import _native as N
        s["cache"] = N.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["batch"] = N.KVBatch(s["table"], s["q_start"], s["kv_len"], s["max_new"], s["max_len"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    case = s["case"]
    if case["op"] == "append":
        return _run_append(s) if own else _plain_append(s)
    if case["op"] == "attend":
        return _run_attend(s) if own else _plain_attend(s)
    return _run_join(s) if own else _plain_join(s)


def _run_append(s):
    from ternary_weight_linear_bit_amd import _native as N
    N.bitnet_kv_append(s["cache"], s["batch"], s["new_k"], s["new_v"], cos=s["cos"], sin=s["sin"],
                       interleaved=s["case"]["pairs"] == "neighbours", q=s["q"], q_out=s["q_out"])
    return {"q": s["q_out"], "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _run_attend(s):
    from ternary_weight_linear_bit_amd import _native as N
    N.bitnet_attention(s["cache"], s["batch"], s["q"], scale=s["softmax_scale"],
                       window=s["case"]["window"], out=s["out"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _run_join(s):
    from ternary_weight_linear_bit_amd import _native as N
    h, x_q, x_scale = N.bitnet_residual_norm(s["y"], s["h"], h_out=s["h_out"], post_weight=s["post"],
                                             gate=s["gate"], scale=s["scale"], pre_weight=s["pre"],
                                             eps=EPS)
    return {"h": h, "x_q": x_q, "x_scale": x_scale}


def _places(s, tokens, page):
    """Of each new token: its sequence, its number there, its position, its page and its slot."""
    start, t = s["q_start"].long(), torch.arange(tokens, device=DEV)
    seq = torch.searchsorted(start, t, right=True) - 1
    number = t - start[seq]
    new = start.diff()
    pos = s["kv_len"].long()[seq] - new[seq] + number
    return seq, number, pos, s["table"].long()[seq, pos // page], pos % page


def _rotate(x, cos, sin, rot, pairs):
    """Rotation of the first `rot` dims by each token's angles, in 32 bits, one rounding per operation."""
    x = x.float()
    a, b = ((x[..., :rot // 2], x[..., rot // 2:rot]) if pairs == "halves" else
            (x[..., 0:rot:2], x[..., 1:rot:2]))
    c, d = cos[:, None, :], sin[:, None, :]
    p, r = a * c - b * d, b * c + a * d
    y = x.clone()
    if pairs == "halves":
        y[..., :rot // 2], y[..., rot // 2:rot] = p, r
    else:
        y[..., 0:rot:2], y[..., 1:rot:2] = p, r
    return y


def _plain_append(s):
    case = s["case"]
    page, tokens = case["page"], s["new_k"].shape[0]
    seq, _, pos, pid, slot = _places(s, tokens, page)
    cos, sin = s["cos"][pos], s["sin"][pos]
    rows = _rotate(s["new_k"], cos, sin, case["rot"], case["pairs"]), s["new_v"].float()
    q = _rotate(s["q"], cos, sin, case["rot"], case["pairs"]).to(s["q"].dtype)
    s["q_out"].copy_(q)
    hk = rows[0].shape[1]
    # the page in which each sequence's new tokens begin, and its slots before them
    new = s["q_start"].long().diff()
    begin = s["kv_len"].long() - new
    first = s["table"].long().gather(1, (begin // page)[:, None].clamp(max=s["table"].shape[1] - 1))[:, 0]
    before = torch.arange(page, device=DEV) < (begin % page)[:, None]          # [seqs, page]
    kept = (new > 0) & (begin % page > 0)
    q127 = torch.full((), 127.0, device=DEV)
    head = torch.arange(hk, device=DEV)
    for name, x in zip(("k", "v"), rows):
        codes, scale = s[name], s[name + "_scale"]
        most = x.abs().amax(-1).clamp(min=1e-5)                                # [tokens, heads]
        top = torch.zeros_like(scale).scatter_reduce(0, pid[:, None].expand(-1, hk), most, "amax")
        need = top / q127
        old = torch.zeros_like(scale)
        old[first] = torch.where(kept[:, None], scale[first], old[first])
        d = torch.where(top > 0, torch.maximum(need, old), scale)
        inv = torch.ones_like(d) / d
        # codes of earlier tokens in those pages, at the new scale
        factor = scale[first] / d[first]                                       # [seqs, heads]
        was = codes[first]
        sel = before[:, None, :, None] if name == "k" else before[:, None, None, :]
        moved = (was.float() * factor[:, :, None, None]).round().to(torch.int8)
        sel = sel & kept[:, None, None, None] & (d[first] > scale[first])[:, :, None, None]
        codes[first] = torch.where(sel, moved, was)
        scale.copy_(d)
        new_codes = (x * inv[pid][:, :, None]).round().clamp(-127, 127).to(torch.int8)
        if name == "k":
            codes[pid[:, None], head[None, :], slot[:, None]] = new_codes
        else:
            codes[pid[:, None], head[None, :], :, slot[:, None]] = new_codes
    return {"q": s["q_out"], "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _plain_attend(s):
    case = s["case"]
    tokens, hq, dim = s["q"].shape
    page, hk, seqs = case["page"], s["k"].shape[1], case["seqs"]
    group, most, table = hq // hk, s["max_new"], s["table"].long()
    seq, number, _, _, _ = _places(s, tokens, page)
    keys = table.shape[1] * page
    k = (s["k"][table].float() * s["k_scale"][table][..., None, None]).transpose(1, 2)
    k = k.reshape(seqs, hk, keys, dim)
    v = (s["v"][table].float() * s["v_scale"][table][..., None, None]).permute(0, 2, 1, 4, 3)
    v = v.reshape(seqs, hk, keys, dim)
    start = s["q_start"].long()
    row = (start[:-1, None] + torch.arange(most, device=DEV)).clamp(max=tokens - 1)
    q = s["q"].float()[row].reshape(seqs, most, hk, group, dim).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(seqs, hk, group * most, dim), k.transpose(2, 3).contiguous())
    x = x.reshape(seqs, hk, group, most, keys).mul_(s["softmax_scale"])
    pos = (s["kv_len"].long() - start.diff())[:, None] + torch.arange(most, device=DEV)
    j = torch.arange(keys, device=DEV)
    seen = j <= pos[..., None]
    if case["window"]:
        seen = seen & (j > pos[..., None] - case["window"])
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x.reshape(seqs, hk, group * most, keys), v)
    out = out.reshape(seqs, hk, group, most, dim) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + total.log())[..., 0]
    out = out.permute(0, 3, 1, 2, 4).reshape(seqs, most, hq, dim)[seq, number]
    lse = lse.permute(0, 3, 1, 2).reshape(seqs, most, hq)[seq, number]
    s["out"].copy_(out)
    s["lse"].copy_(lse)
    return {"out": s["out"], "lse": s["lse"]}


def _plain_norm(x, weight):
    """RN32(RN32(x r) w); the mean of squares is summed in 64 bits and rounded once."""
    ms = x.double().square().mean(-1, keepdim=True).float()
    r = ((ms + torch.full_like(ms, EPS)).double().sqrt().reciprocal()).float()
    return (x * r) * weight


def _plain_join(s):
    z = s["y"].float()
    if s["post"] is not None:
        z = _plain_norm(z, s["post"])
    if s["gate"] is not None:
        z = z * s["gate"].float()
    h = (s["h"].float() + z * s["scale"]).to(s["h"].dtype)
    s["h_out"].copy_(h)
    u = _plain_norm(h.float(), s["pre"])
    most = u.abs().amax(-1).clamp(min=1e-5)
    q127 = torch.full_like(most, 127.0)
    x_q = (u * (q127 / most)[:, None]).round().clamp(-128, 127).to(torch.int8)
    return {"h": s["h_out"], "x_q": x_q, "x_scale": most / q127}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "join": _exact_join}[case["op"]](s)


def _r(x):
    """Where the definition rounds to 32 bits."""
    return x.float().double()


def _exact_append(s):
    """Codes follow the definition's roundings; scales and rotated queries are in 64 bits throughout."""
    case = s["case"]
    page, rot, half = case["page"], case["rot"], case["rot"] // 2
    new, length, tokens, _ = _lengths(case)
    if case["pairs"] == "halves":
        ia, ib = torch.arange(half, device=DEV), torch.arange(half, device=DEV) + half
    else:
        ia, ib = torch.arange(half, device=DEV) * 2, torch.arange(half, device=DEV) * 2 + 1
    pos = torch.cat([torch.arange(ln - n, ln, device=DEV) for n, ln in zip(new, length)])
    c, d = s["cos"][pos].double()[:, None], s["sin"][pos].double()[:, None]

    def turned(x, r):
        x = x.double()
        y = x.clone()
        y[..., ia] = r(r(x[..., ia] * c) - r(x[..., ib] * d))
        y[..., ib] = r(r(x[..., ib] * c) + r(x[..., ia] * d))
        return y

    q = turned(s["q"], lambda x: x)
    rows = {"k": turned(s["new_k"], _r), "v": s["new_v"].double()}
    codes = {"k": s["k"].clone(), "v": s["v"].transpose(2, 3).clone()}
    scales = {n: s[n + "_scale"].double() for n in rows}
    table, t0 = s["table"].tolist(), 0
    for b, (n, ln) in enumerate(zip(new, length)):
        p, end = ln - n, t0 + n
        while t0 < end:
            pid, lo = table[b][p // page], p % page
            m = min(page - lo, end - t0)
            for name, x in rows.items():
                part = x[t0:t0 + m].transpose(0, 1)                         # [heads, m, dim]
                need = part.abs().amax((1, 2)).clamp(min=float(torch.tensor(1e-5))) / 127
                old = scales[name][pid]
                to = torch.maximum(need, old) if lo else need
                f = _r(_r(old) / _r(to))[:, None, None]
                grown = (_r(to) > _r(old))[:, None, None]
                kept = codes[name][pid][:, :lo]
                codes[name][pid][:, :lo] = torch.where(
                    grown, _r(kept.double() * f).round().to(torch.int8), kept)
                inv = _r(1 / _r(to))[:, None, None]
                codes[name][pid][:, lo:lo + m] = _r(part * inv).round().clamp(-127, 127).to(torch.int8)
                scales[name][pid] = to
            p, t0 = p + m, t0 + m
    return {"q": q, "k": codes["k"], "v": codes["v"].transpose(2, 3).contiguous(),
            "k_scale": scales["k"], "v_scale": scales["v"]}


def _exact_attend(s):
    case = s["case"]
    new, length, tokens, _ = _lengths(case)
    hq, hk, dim = HEADS[case["shape"]]
    group, page = hq // hk, case["page"]
    out = torch.zeros(tokens, hq, dim, dtype=torch.float64, device=DEV)
    lse = torch.zeros(tokens, hq, dtype=torch.float64, device=DEV)
    t0 = 0
    for b, (n, ln) in enumerate(zip(new, length)):
        ids = s["table"][b, :-(-ln // page)].long()
        pos = torch.arange(ln - n, ln, device=DEV)[:, None]
        j = torch.arange(ln, device=DEV)
        hidden = (j > pos) | ((j <= pos - case["window"]) if case["window"] else (j < 0))
        for h in range(hk):
            k = (s["k"][ids, h].double() * s["k_scale"][ids, h].double()[:, None, None]).reshape(-1, dim)[:ln]
            v = (s["v"][ids, h].double() * s["v_scale"][ids, h].double()[:, None, None])
            v = v.transpose(1, 2).reshape(-1, dim)[:ln]
            for g in range(h * group, (h + 1) * group):
                x = (s["q"][t0:t0 + n, g].double() @ k.T) * s["softmax_scale"]
                x.masked_fill_(hidden, -math.inf)
                at = torch.logsumexp(x, -1)
                lse[t0:t0 + n, g] = at
                out[t0:t0 + n, g] = (x - at[:, None]).exp() @ v
        t0 += n
    return {"out": out, "lse": lse}


def _exact_join(s):
    """Each rounding of the definition is made by itself, from a value in 64 bits."""
    eps = float(torch.tensor(EPS))

    def norm(x, w):
        ms = _r((x * x).sum(-1, keepdim=True) / x.shape[-1])
        return _r(_r(x * _r(1 / _r(ms + eps).sqrt())) * w.double())

    z = s["y"].double()
    if s["post"] is not None:
        z = norm(z, s["post"])
    if s["gate"] is not None:
        z = _r(z * s["gate"].double())
    h = _r(s["h"].double() + _r(z * s["scale"])).to(s["h"].dtype).double()
    u = norm(h, s["pre"])
    most = u.abs().amax(-1).clamp(min=float(torch.tensor(1e-5)))
    x_q = _r(u * _r(127 / most)[:, None]).round().clamp(-128, 127).to(torch.int8)
    return {"h": h, "x_q": x_q, "x_scale": most / 127}
