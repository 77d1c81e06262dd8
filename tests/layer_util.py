"""Inputs, and bounds on attention's error, shared by the cache and attention tests."""

import numpy as np

F32 = np.float32


def seqs(news, lens, page, spare=2, seed=0, width=None):
    """q_start, kv_len and a page table whose pages are shuffled; ids never used: -1."""
    rng = np.random.default_rng(seed)
    q_start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    counts = [(n + page - 1) // page for n in lens]
    width = max(max(counts), 1) if width is None else width
    pages = sum(counts) + spare
    order = rng.permutation(pages)
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    return q_start, np.asarray(lens, np.int32), table, pages


def cache(pages, heads, page, dim, seed=0):
    """Random codes and scales (k, v, k_scale, v_scale)."""
    rng = np.random.default_rng(seed)
    k = rng.integers(-127, 128, (pages, heads, page, dim)).astype(np.int8)
    v = rng.integers(-127, 128, (pages, heads, dim, page)).astype(np.int8)
    ks = np.exp(rng.normal(0, 0.5, (pages, heads))).astype(F32) * F32(3 / 127)
    vs = np.exp(rng.normal(0, 0.5, (pages, heads))).astype(F32) * F32(3 / 127)
    return k, v, ks, vs


def tables(positions, rot):
    inv = 10000.0 ** (-np.arange(rot // 2) * 2.0 / rot)
    a = np.arange(positions)[:, None] * inv
    return np.cos(a).astype(F32), np.sin(a).astype(F32)


def attention_bounds(out, lse, absv, flat, top, reach, q, keys, exact_io):
    """How far the kernel's out and lse may be from the float64 ones, elementwise.

    The queries enter the products with an error of at most 2^-22 of the row's largest
    |q| (bf16 ones exactly, where they are not below 2^-14 of it), which moves a logit by
    at most reach * max|q| * 2^-22.  Weights w = p dv are kept to 2^-b of the row's
    largest (b = 15.9: two 8-bit digits, 127 * 256 steps; fp32 in and out: 22), or, for
    bf16, rounded to 11 bits each (2^-11 of sum w|v|).  Fp32 arithmetic: a logit within
    2^-21 of the largest |s| (a few roundings), exp within 2^-20, sums over `keys` keys
    within (keys / 16 + 32) 2^-24 of sum w|v|.  A logit error e moves every weight by a
    factor within exp(2e) after the division.  lse has the logits' errors and the sum's,
    whatever the output's type.  bf16 outputs are rounded: 2^-8 of the value (half a step)."""
    b = 22.0 if exact_io else 15.9
    amax = np.abs(q).max(-1)
    e = reach * amax * 2.0 ** -22 + top * 2.0 ** -21 + 2.0 ** -20
    rel = np.expm1(2 * e) + (keys / 16 + 32) * 2.0 ** -24
    tol = rel[..., None] * absv + flat * 2.0 ** -b     # flat: summed over the visible keys
    if not exact_io:
        tol = tol + 2.0 ** -11 * absv + 2.0 ** -8 * np.abs(out)
    else:
        tol = tol + 2.0 ** -24 * np.abs(out)
    tol_lse = np.where(np.isfinite(lse), e + (keys / 16 + 32) * 2.0 ** -24
                       + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0)), 0)
    return tol + 1e-30, tol_lse
