"""Rows in which few keys outweigh the others, and bounds that look at each weight by
itself: what a trained model's heads are like, and what random queries and keys are not."""

import numpy as np

F32 = np.float32
REACH = 2.0 ** -48   # weights below this share of their row's largest may count as 0


def peaked(rng, rows, q_heads, heads, dim, keys, gap, at, value=(True,), spread=1.0, noise=0.02):
    """Queries fp32 [rows, q_heads, dim] (bf16 values), and for each kv head key and value codes
    [heads, keys, dim], the page scale of keys, of values, and the softmax scale.

    The logits of most keys are N(0, spread^2); query head i has a key at position at + i whose
    logit lies about `gap` above the highest of them.  value: whether those keys have values, head
    by head in turn."""
    group = q_heads // heads
    base = rng.standard_normal((q_heads, dim))
    q = base + noise * rng.standard_normal((rows, q_heads, dim))
    q = bf16(q)
    sigma = 10.0
    kc = np.clip(np.rint(rng.normal(0, sigma, (heads, keys, dim))), -127, 127)
    vc = np.clip(np.rint(rng.normal(20, 40, (heads, keys, dim))), -127, 127)
    dk, dv = F32(1 / 64), F32(3 / 127)
    scale = F32(spread / (sigma * float(dk) * dim ** 0.5))
    for i in range(q_heads):
        h, j = i // group, (at + i) % keys
        # |q|^2 near dim: a logit of scale dk a |q|^2 from codes a q
        far = spread * np.sqrt(2 * np.log(max(keys, 3))) + gap
        a = far / (float(scale) * float(dk) * (base[i] ** 2).sum())
        kc[h, j] = np.clip(np.rint(a * base[i]), -127, 127)
        if not value[i % len(value)]:
            vc[h, j] = 0
    return q, kc.astype(np.int8), vc.astype(np.int8), dk, dv, scale


def bf16(x):
    """Values of bf16 nearest to x (ties to even), as fp32."""
    u = np.ascontiguousarray(x, F32).view(np.uint32)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & np.uint32(0xFFFF0000)
    return u.view(F32)


def paged(kc, vc, page):
    """Codes [heads, keys, dim] as pages: k [pages, heads, page, dim], v [pages, heads, dim, page];
    what lies behind the last key is not zero."""
    heads, keys, dim = kc.shape
    n = -(-keys // page)
    k = np.full((heads, n * page, dim), 101, np.int8)
    v = np.full((heads, n * page, dim), -99, np.int8)
    k[:, :keys], v[:, :keys] = kc, vc
    k = k.reshape(heads, n, page, dim).transpose(1, 0, 2, 3)
    v = v.reshape(heads, n, page, dim).transpose(1, 0, 3, 2)
    return np.ascontiguousarray(k), np.ascontiguousarray(v)


def one_key_a_dim(rng, keys, dim, heads, but=None):
    """Value codes [heads, keys, dim] of which each dim has one key only (127), none of head h's
    but[h], so that an output is that key's weight."""
    vc = np.zeros((heads, keys, dim), np.int8)
    for h in range(heads):
        some = np.setdiff1d(np.arange(keys), but[h] if but else ())
        vc[h, rng.choice(some, dim, replace=len(some) < dim), np.arange(dim)] = 127
    return vc


def weight_bounds(out, lse, absv, flat, top, reach, q, keys, exact_io, out_bf16, steps=0):
    """How far out and lse may be from the float64 ones, elementwise, whatever the values are.

    A logit is off by at most e (layer_util.attention_bounds: the queries to 2^-22 of their row's
    largest, fp32 roundings 2^-21 of the largest |s|, exp 2^-20), which moves every weight by a
    factor within exp(2 e) after the division.  Each weight keeps 11 bits, 22 with fp32 in and
    out: it is off by at most 2^-11 or 2^-22 of itself, and the sum of w v by that share of the
    sum of w |v|.  fp32 sums over `keys` keys: (keys / 16 + 32) 2^-24 of it.  Weights below
    2^-48 of the row's largest may be 0: flat (the largest weight times the sum of |v|)
    times 2^-48.  In each of `steps` steps (the prompt kernel) the weights may further lack what
    moves no sum by more than 2^-24 of the row's largest sum of w |v|.  The output's type rounds
    by half a step: 2^-8 (bf16) or 2^-24 of the value."""
    e = reach * np.abs(q).max(-1) * 2.0 ** -22 + top * 2.0 ** -21 + 2.0 ** -20
    sums = (keys / 16 + 32) * 2.0 ** -24
    held = 2.0 ** -22 if exact_io else 2.0 ** -11
    err = (np.expm1(2 * e) + sums + held)[..., None] * absv + flat * REACH
    err = err + (steps * 2.0 ** -24 * absv.max(-1))[..., None]
    half = 2.0 ** -8 if out_bf16 else 2.0 ** -24
    tol_lse = e + sums + 2.0 ** -22 * np.abs(lse)
    return err + half * (np.abs(out) + err) + 1e-30, tol_lse
