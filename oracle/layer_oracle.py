"""CPU oracle of what lies between a layer's ternary products: the paged 8-bit
cache of keys and values, attention over it, and the join with the residual
stream.  Plain numpy, written from the definitions; shares no code with the HIP
path.

The pages name the parts and give no formulas (communeify.com, section on BitNet
b1.58 2B4T, architecture item: rotary position embeddings, subln normalisation, no
biases).  Readings:

K1  rotation of a pair (a, b) with cosine c and sine s (fp32 tables of the caller):
    (RN32(RN32(a c) - RN32(b s)), RN32(RN32(b c) + RN32(a s))).
K2  a page of one head has one scale.  Rows x that a call adds to it (all of them
    together): need = RN32(max(max|x|, RN32(1e-5)) / 127).  A page whose slot 0 is
    written takes d' = need, another d' = max(d, need).
K3  new codes clip(rne(RN32(x * RN32(1/d'))), -127, 127); with d' > d earlier codes c
    become rne(RN32(c * RN32(d/d'))).
K4  attention in float64: s = scale dk (q . kc) over the visible keys,
    out = sum e^(s-m) dv vc / sum e^(s-m), lse = m + ln sum; a row without keys: 0, -inf.
J1  z = RN32(RN32(y r) w) (norm behind the block) or y; z = RN32(z gate);
    h' = RN(RN32(h + RN32(z scale))) in the stream's type; u = RN32(RN32(h' r) w) (norm
    before the next block) or h'; codes as O4 forms them.  r as in N2.
"""

from __future__ import annotations

import numpy as np

from oracle import bitnet_oracle as O

F32 = np.float32


def rotate(x, cos, sin, interleaved):
    """K1 on x [..., D] fp32 with cos / sin [rot/2]: dims from rot on pass through."""
    x = np.asarray(x, F32)
    half = len(cos)
    y = x.copy()
    if half == 0:
        return y
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + (1 if interleaved else half)
    a, b = x[..., ia], x[..., ib]
    c, s = np.asarray(cos, F32), np.asarray(sin, F32)
    y[..., ia] = (a * c).astype(F32) - (b * s).astype(F32)
    y[..., ib] = (b * c).astype(F32) + (a * s).astype(F32)
    return y


def page_scale(x, old):
    """K2: scale of a page with new rows x; old: its scale, or None where it begins."""
    need = F32(max(F32(np.abs(x).max()), O.EPS)) / O.QB
    return need if old is None else max(F32(old), need)


def append_page(codes, scale, rows, lo):
    """K2 and K3 on one page of one head: codes int8 [P, D] (changed), its scale, new
    fp32 rows [n, D] at slots lo ..; returns the new scale."""
    d = page_scale(rows, None if lo == 0 else scale)
    if lo > 0 and d > scale:
        f = F32(scale) / d
        codes[:lo] = np.rint((codes[:lo].astype(F32) * f).astype(F32)).astype(np.int8)
    inv = F32(1.0) / d
    q = np.rint((rows * inv).astype(F32))
    codes[lo:lo + len(rows)] = np.clip(q, -127, 127).astype(np.int8)
    return d


def spans(q_start, kv_len, tokens, max_new, max_len):
    """Per sequence: (first row, rows, position of the first row, cached tokens)."""
    out = []
    for b in range(len(kv_len)):
        s0 = min(max(int(q_start[b]), 0), tokens)
        n = min(max(int(q_start[b + 1]), s0), tokens) - s0
        ln = min(max(int(kv_len[b]), 0), max_len)
        out.append((s0, n, ln - n, ln))
    return out


def kv_append(k, v, k_scale, v_scale, table, q_start, kv_len, new_k, new_v, cos=None, sin=None,
              interleaved=False, q=None, max_new=None, max_len=None):
    """The cache arrays ([pages, heads, P, D], v [pages, heads, D, P]) after an append, and
    the rotated queries in fp32 (rows outside every sequence: NaN).  Inputs are not changed."""
    k, v, ks, vs = k.copy(), v.copy(), k_scale.copy(), v_scale.copy()
    pages, heads, P, D = k.shape
    T = new_k.shape[0]
    max_new = T if max_new is None else max_new
    max_len = table.shape[1] * P if max_len is None else max_len
    none = np.zeros(0, F32)
    q_out = None if q is None else np.full(q.shape, np.nan, F32)
    for b, (s0, n, first, ln) in enumerate(spans(q_start, kv_len, T, max_new, max_len)):
        by_page = {}
        for i in range(min(n, max_new)):
            pos = first + i
            c, s = (none, none) if cos is None or pos < 0 else (cos[pos], sin[pos])
            if q is not None:
                q_out[s0 + i] = rotate(q[s0 + i], c, s, interleaved)
            if pos >= 0:
                by_page.setdefault(pos // P, []).append(
                    (pos % P, rotate(new_k[s0 + i], c, s, interleaved), new_v[s0 + i]))
        for pg, rows in by_page.items():
            pid = int(table[b, pg])
            if not 0 <= pid < pages:
                continue
            lo = rows[0][0]
            for h in range(heads):
                ks[pid, h] = append_page(k[pid, h], ks[pid, h],
                                         np.stack([r[1][h] for r in rows]).astype(F32), lo)
                page_v = v[pid, h].T.copy()
                vs[pid, h] = append_page(page_v, vs[pid, h],
                                         np.stack([r[2][h] for r in rows]).astype(F32), lo)
                v[pid, h] = page_v.T
    return k, v, ks, vs, q_out


def gather(codes_k, codes_v, k_scale, v_scale, table_row, head, length):
    """float64 keys, values [length, D], the value codes and scales, and which keys exist."""
    pages, _, P, D = codes_k.shape
    ids = np.asarray(table_row[:(length + P - 1) // P], np.int64)
    ok = (ids >= 0) & (ids < pages)
    safe = np.where(ok, ids, 0)
    dk = np.where(ok, k_scale[safe, head], 0).astype(np.float64)
    dv = np.where(ok, v_scale[safe, head], 0).astype(np.float64)
    kc = codes_k[safe, head].astype(np.float64)
    vc = codes_v[safe, head].transpose(0, 2, 1).astype(np.float64)
    rep = lambda x: np.repeat(x, P)[:length]
    return (kc.reshape(-1, D)[:length], vc.reshape(-1, D)[:length], rep(dk), rep(dv), rep(ok))


def attention(k, v, k_scale, v_scale, table, q_start, kv_len, q, scale, window=0, max_new=None,
              max_len=None, detail=False):
    """K4 in float64: (out [T, Hq, D], lse [T, Hq]); rows outside every sequence are NaN.

    With detail also what error bounds need: sum w|v| [T, Hq, D]; the sum over the
    visible keys of |vc| times the largest e^(s-m) dv, over sum e^(s-m) [T, Hq, D]; the
    largest |s| [T, Hq]; and the largest scale dk sum_d |kc| [T, Hq]."""
    T, Hq, D = q.shape
    P, heads = k.shape[2], k.shape[1]
    group = Hq // heads
    max_new = T if max_new is None else max_new
    max_len = table.shape[1] * P if max_len is None else max_len
    out = np.full((T, Hq, D), np.nan)
    lse = np.full((T, Hq), np.nan)
    absv, flat = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    top, reach = np.zeros((T, Hq)), np.zeros((T, Hq))
    for b, (s0, n, first, ln) in enumerate(spans(q_start, kv_len, T, max_new, max_len)):
        for h in range(heads):
            kc, vc, dk, dv, ok = gather(k, v, k_scale, v_scale, table[b], h, ln)
            rows = min(n, max_new)
            if rows == 0:
                continue
            pos = first + np.arange(rows)[:, None]
            j = np.arange(ln)[None, :]
            seen = ok[None, :] & (j <= pos)
            if window:
                seen &= j > pos - window
            some = seen.any(1)
            t = slice(s0, s0 + rows)
            for g in range(h * group, (h + 1) * group):
                out[t, g], lse[t, g] = 0.0, -np.inf
                if not some.any():
                    continue
                with np.errstate(invalid="ignore", over="ignore"):   # scales of pages nobody sees
                    s = scale * dk * (q[t, g].astype(np.float64) @ kc.T)
                s = np.where(seen, s, -np.inf)
                m = np.where(some, s.max(1), 0.0)[:, None]
                w = np.exp(s - m)
                total = np.where(some, w.sum(1), 1.0)[:, None]
                lse[t, g] = np.where(some, (m + np.log(total))[:, 0], -np.inf)
                w = np.where(seen, w * np.where(seen.any(0), dv, 0.0), 0.0)
                out[t, g] = (w @ vc) / total
                if detail:
                    absv[t, g] = (w @ np.abs(vc)) / total
                    flat[t, g] = w.max(1)[:, None] * (seen @ np.abs(vc)) / total
                    top[t, g] = np.where(seen, np.abs(s), 0.0).max(1)
                    reach[t, g] = np.where(seen, abs(scale) * dk * np.abs(kc).sum(1), 0.0).max(1)
    return (out, lse, absv, flat, top, reach) if detail else (out, lse)


def residual_norm(y, h, h_bf16=False, post_weight=None, gate=None, scale=1.0, pre_weight=None,
                  eps=1e-5):
    """J1: (h' fp32 values of the stream's type, u fp32, codes, scales); gate [K] or [M, K]."""
    z = np.ascontiguousarray(y, F32)
    if post_weight is not None:
        z = O.rms_normalise(z, post_weight, eps)
    if gate is not None:
        z = (z * np.asarray(gate, F32)).astype(F32)
    h2 = (np.asarray(h, F32) + (z * F32(scale)).astype(F32)).astype(F32)
    if h_bf16:
        h2 = O.bf16_bits_to_f32(O.f32_to_bf16_bits(h2))
    u = h2 if pre_weight is None else O.rms_normalise(h2, pre_weight, eps)
    xq, d = O.quantize_acts(u)
    return h2, u, xq, d
