"""CPU oracle of a feed-forward of ternary experts: routing, products grouped by expert with
what follows them, and the combination.  Plain numpy, written from the definitions; shares no
code with the HIP path.

The pages describe dense layers only (the products and their rescale: dashen-tech.com, "BitNet.cpp
深度解析", section 3.1); readings for the rest:

E1  choice: a token's topk largest logits, ties lowest index first; -inf and NaN are never chosen
    (expert -1, weight 0 where fewer are left).
E2  weight: scale times the softmax of the chosen logit among all of them ("softmax"), among the
    chosen ones ("chosen"), or 1 / (1 + e^-x) ("sigmoid"), in 64 bits; logits that equal the
    largest count e^0.
E3  plan: pairs p = m topk + j that have an expert, sorted by (expert, p); a pair's place is its slot.
E4  product: v = RN32(float(acc) RN32(gamma d)), v = RN32(v + b), a = act(v), a = RN32(a u),
    a = RN32(a + residual); relu2 = RN32(max(v, 0)^2); silu and gelu in 64 bits.
E5  combination: from the residual (or 0), RN32(out + RN32(weight y)) over j ascending.
"""

from __future__ import annotations

import math

import numpy as np

from oracle import bitnet_oracle as O

F32 = np.float32


def choose(logits, topk):
    """E1 on logits [tokens, experts]: expert int32 [tokens, topk]."""
    x = np.asarray(logits, np.float64)
    out = np.full((x.shape[0], topk), -1, np.int32)
    for m, row in enumerate(x):
        able = [e for e in range(len(row)) if row[e] > -np.inf]        # False for NaN
        able.sort(key=lambda e: (-row[e], e))
        able = able[:topk]
        out[m, :len(able)] = able
    return out


def weigh(logits, expert, score, scale):
    """E2 in float64: weight [tokens, topk]."""
    x = np.asarray(logits, np.float64)
    out = np.zeros(expert.shape)
    for m, row in enumerate(x):
        chosen = [int(e) for e in expert[m] if e >= 0]
        if not chosen:
            continue
        top = row[chosen[0]]

        def power(z):
            return 1.0 if z == top else math.exp(z - top)
        if score == "sigmoid":
            w = [1.0 / (1.0 + math.exp(-row[e])) if row[e] > -700 else 0.0 for e in chosen]
        else:
            over = chosen if score == "chosen" else [e for e in range(len(row)) if row[e] > -np.inf]
            total = math.fsum(power(row[e]) for e in over)
            w = [power(row[e]) / total for e in chosen]
        out[m, :len(chosen)] = np.asarray(w) * float(F32(scale))
    return out


def plan(expert, experts):
    """E3: offset [experts + 1], pair [pairs], slot like expert."""
    flat = np.asarray(expert).reshape(-1)
    lists = [[p for p, e in enumerate(flat.tolist()) if e == x] for x in range(experts)]
    offset = np.cumsum([0] + [len(v) for v in lists]).astype(np.int32)
    pair = np.full(flat.size, -1, np.int32)
    slot = np.full(flat.size, -1, np.int32)
    for s, p in enumerate(p for v in lists for p in v):
        pair[s], slot[p] = p, s
    return offset, pair, slot.reshape(np.shape(expert))


def accumulate(q, x_q):
    """Exact integer products of x_q [rows, K] with ternary q [N, K] (exact in float64)."""
    return np.asarray(x_q, np.float64) @ np.asarray(q, np.float64).T


def linear(q, gamma, x_q, d, bias=None):
    """v of E4."""
    acc = accumulate(q, x_q).astype(F32)
    s = (F32(gamma) * np.asarray(d, F32)).astype(F32)
    v = (acc * s[:, None]).astype(F32)
    return v if bias is None else (v + np.asarray(bias, F32)).astype(F32)


def phi(v):
    """The standard normal distribution function, float64."""
    return np.vectorize(lambda z: 0.5 * math.erfc(-z * math.sqrt(0.5)), otypes=[np.float64])(v)


def activate(v, act):
    """act(v): fp32 for none and relu2, float64 for the others."""
    if act == "relu2":
        a = np.maximum(v, F32(0))
        with np.errstate(over="ignore"):
            return (a * a).astype(F32)
    z = np.asarray(v, np.float64)
    if act == "silu":
        e = np.exp(-np.abs(z))
        return np.where(z < 0, z * e, z) / (1 + e)
    if act == "gelu":
        return z * phi(z)
    return v


def product(q, gamma, x_q, d, bias=None, act="none", up=None, residual=None):
    """E4 before the last rounding; up: (q, gamma, bias).  Returns (a, tol): a fp32 and tol None
    where the definition is exact, else float64 with the bound that silu's and gelu's errors
    (2^-20 of the value, gelu 2^-24 of |v| beside it) and the roundings of the gating and the
    residual (2^-24 of the result each) leave, and a subnormal's half step, 2^-150, for each rounding."""
    v = linear(q, gamma, x_q, d, bias)
    a = activate(v, act)
    u = None if up is None else linear(up[0], up[1], x_q, d, up[2])
    if act in ("none", "relu2"):
        if u is not None:
            a = (a * u).astype(F32)
        if residual is not None:
            a = (a + np.asarray(residual, F32)).astype(F32)
        return a, None
    tol = 2.0 ** -20 * np.abs(a) + (2.0 ** -24 * np.abs(np.float64(v)) if act == "gelu" else 0) + 2.0 ** -149
    if u is not None:
        tol = tol * np.abs(np.float64(u)) + 2.0 ** -24 * np.abs(a * u) + 2.0 ** -150
        a = a * u
    if residual is not None:
        a = a + np.asarray(residual, np.float64)
        tol = tol + 2.0 ** -24 * np.abs(a)
    return a, tol + 2.0 ** -24 * np.abs(a)


def combine(weight, slot, y, residual=None):
    """E5 before the last rounding, fp32 [tokens, K]."""
    m, topk = slot.shape
    out = np.zeros((m, y.shape[1]), F32) if residual is None else np.asarray(residual, F32).copy()
    for t in range(m):
        for j in range(topk):
            s = slot[t, j]
            if 0 <= s < y.shape[0]:
                out[t] = out[t] + (F32(weight[t, j]) * np.asarray(y[s], F32)).astype(F32)
    return out


def bf16(x):
    """fp32 values rounded to bf16, as fp32."""
    return O.bf16_bits_to_f32(O.f32_to_bf16_bits(np.asarray(x, F32)))
