"""The arithmetic of the attention kernels' weights, step by step on the CPU, on rows in which one
key outweighs thousands; and that the bounds of such rows reject what loses the small
weights."""

import numpy as np
import pytest

from oracle import layer_oracle as L
from attention_rows import REACH, one_key_a_dim, paged, peaked, weight_bounds

F32 = np.float32
STEP, WAVES, LIFT, MAGIC = 64, 4, 14, F32(1.5 * 2.0 ** 23 + 128)


def reference(q, kc, vc, dk, dv, scale, keys):
    """L.attention of one row of one head, with what the bounds need."""
    k, v = paged(kc[None], vc[None], 64)
    n = len(k)
    ks, vs = np.full((n, 1), dk, F32), np.full((n, 1), dv, F32)
    return L.attention(k, v, ks, vs, np.arange(n, dtype=np.int32)[None], [0, 1], [keys], q[None, None], scale,
                       detail=True)


def digits(y, unit):
    """Two signed base-256 digits of round(y / unit), as the kernel takes them from the bits of one
    sum, and what is left of y."""
    t = (y + MAGIC * unit).astype(F32)
    u = t.view(np.uint32)
    lo = ((u & 0xFF) ^ 0x80).astype(np.uint8).view(np.int8)
    hi = ((u >> 8) & 0xFF).astype(np.uint8).view(np.int8)
    hi, lo = hi.astype(np.int64), lo.astype(np.int64)
    rest = (y - (t - MAGIC * unit)).astype(F32)
    np.testing.assert_array_equal(hi * 256 + lo, np.rint(y.astype(np.float64) / unit))
    np.testing.assert_array_equal(rest, y.astype(np.float64) - (hi * 256 + lo) * float(unit))
    return hi, lo, rest


def by_steps(q, kc, vc, dk, dv, scale, bits):
    """The kernel's sums of one row: each wave takes every fourth step of 64 keys, weights in
    digits against the step's own reference, pass after pass until each keeps `bits` bits."""
    keys, dim = kc.shape
    s = (kc.astype(np.float64) @ q.astype(np.float64)).astype(F32)
    ck, lv = F32(scale * F32(dk) * F32(np.log2(np.e))), F32(np.log2(dv))
    x = (s * ck).astype(F32) + lv
    parts = []
    for w in range(WAVES):
        m, r = F32(-np.inf), F32(0)
        o, l = np.zeros(dim, F32), F32(0)
        for at in range(w * STEP, keys, WAVES * STEP):
            xs, vs = x[at:at + STEP], vc[at:at + STEP].astype(np.int64)
            mx = xs.max()
            m = max(m, mx)
            to = max(np.ceil(mx), np.ceil(m) - 49) - F32(LIFT)
            alpha = F32(2.0 ** float(np.clip(r - to, -200, 126)))
            r = to
            p = np.exp2(xs - to).astype(F32)
            l = F32(l * alpha + F32(p.sum(dtype=F32) * (F32(1) / dv)))
            floor = F32(2.0 ** float(np.ceil(m) - 49 - r))
            low = p[p >= floor].min()
            y, unit, o = p, F32(1), (o * alpha).astype(F32)
            while True:
                hi, lo, y = digits(y, unit)
                o = (o + (hi @ vs * 256 + lo @ vs).astype(F32) * unit).astype(F32)
                if low >= unit * 2 ** (bits - 1):
                    break
                unit = unit * F32(2.0 ** -15)
        if np.isfinite(m):
            parts.append((r, l, o))
    top = max(p[0] for p in parts)
    return sum(p[2] * 2.0 ** float(p[0] - top) for p in parts) / sum(p[1] * 2.0 ** float(p[0] - top) for p in parts)


def fixed_reference(q, kc, vc, dk, dv, scale, top):
    """Weights as integers of `top` steps against each wave's running maximum."""
    x = scale * dk * (kc.astype(np.float64) @ q.astype(np.float64))
    o, l = 0.0, 0.0
    for w in range(WAVES):
        m = -np.inf
        for at in range(w * STEP, len(kc), WAVES * STEP):
            m = max(m, x[at:at + STEP].max())
            p = np.exp(x[at:at + STEP] - m)
            f = np.exp(m - x.max())
            l += p.sum() * f
            o = o + np.rint(p * top) / top @ vc[at:at + STEP] * f * dv
    return o / l


def a_row(keys, gap, value=False, seed=0, at=0):
    rng = np.random.default_rng(seed)
    q, kc, vc, dk, dv, scale = peaked(rng, 1, 1, 1, 128, keys, gap, at, (value,))
    return q[0, 0], kc[0], vc[0], dk, dv, scale


def bounds_of(row, exact_io, out_bf16):
    q, kc, vc, dk, dv, scale = row
    want, lse, *detail = reference(*row, len(kc))
    tol, _ = weight_bounds(want, lse, *detail, q[None, None], np.full(lse.shape, float(len(kc))), exact_io,
                           out_bf16)
    return want[0, 0], tol[0, 0]


@pytest.mark.parametrize("keys", [64, 1024, 8191])
@pytest.mark.parametrize("gap", [0, 6, 9, 12, 14, 18, 30])
@pytest.mark.parametrize("bits", [11, 22])
def test_steps_keep_small_weights(keys, gap, bits):
    for value, at in ((False, 0), (True, keys // 2), (False, keys - 1)):
        row = a_row(keys, gap, value, seed=keys + gap, at=at)
        want, tol = bounds_of(row, bits == 22, False)
        got = by_steps(*row, bits)
        assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)


@pytest.mark.parametrize("spread", [0.3, 1.5, 5.0, 9.0])
@pytest.mark.parametrize("bits", [11, 22])
def test_each_weight_by_itself(spread, bits):
    """Every dim has the value of one key only: its output is that key's weight."""
    rng = np.random.default_rng(7)
    q, kc, _, dk, dv, scale = peaked(rng, 1, 1, 1, 128, 300, 5, 40, spread=spread)
    vc = one_key_a_dim(rng, 300, 128, 1)
    row = (q[0, 0], kc[0], vc[0], dk, dv, scale)
    want, tol = bounds_of(row, bits == 22, False)
    got = by_steps(*row, bits)
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)


@pytest.mark.parametrize("keys", [1024, 4096, 8191])
@pytest.mark.parametrize("gap", [9, 10.5, 12, 14])
def test_bounds_reject_lost_weights(keys, gap):
    """What must not pass on such rows: nothing at all, the small weights left out, and weights of
    15 bits against the running maximum (of 23 where 22 bits of each are kept)."""
    row = a_row(keys, gap, seed=3)
    q, kc, vc, dk, dv, scale = row
    for exact_io, out_bf16 in ((False, True), (False, False), (True, False)):
        want, tol = bounds_of(row, exact_io, out_bf16)
        assert np.mean(np.abs(want) > tol) > 0.9                     # an output of zeros
        x = scale * dk * (kc.astype(np.float64) @ q.astype(np.float64))
        w = np.exp(x - x.max())
        none = np.where(w < 2.0 ** -13, 0, w) @ vc * dv / w.sum()     # small weights left out
        assert gap < 12 or np.mean(np.abs(none - want) > tol) > 0.9
        old = fixed_reference(*row, 8323072.0 if exact_io else 32512.0)
        if not exact_io or gap >= 12:
            assert np.mean(np.abs(old - want) > tol) > 0.2


def test_floor_is_small():
    """All the weights that may count as 0, of 2^24 keys, are less than half of fp32's last bit."""
    assert REACH * 2 ** 24 <= 2.0 ** -24


@pytest.mark.parametrize("terms,lift,held,up", [(1, 7, -14, 29), (2, 14, -3, 33)])
def test_prompt_terms_hold_small_weights(terms, lift, held, up):
    """The prompt kernel's fp16 terms of a weight, and of what they lack where it is below
    2^held: 11 bits a term down to 2^-48 of the largest; without them a sum over 64 keys of codes
    up to 127 lacks at most 2^-12."""
    rng = np.random.default_rng(5)

    def split(x):
        out, rest = np.zeros_like(x), x
        for _ in range(terms):
            t = rest.astype(np.float16).astype(F32)
            out, rest = out + t.astype(np.float64), (rest - t).astype(F32)
        return out, rest
    p = np.exp2(rng.uniform(lift - 48, 15, 100000)).astype(F32)
    first, rest = split(p)
    assert np.all(np.isfinite(first))
    np.testing.assert_array_equal(first + rest, p)                # nothing is lost on the way
    small = p < 2.0 ** held
    assert np.all(np.abs(rest[~small]) <= 2.0 ** (-11 * terms) * p[~small])
    assert 64 * 127 * np.abs(rest[small]).max() <= 2.0 ** -12
    second, _ = split((rest[small] * F32(2.0 ** up)).astype(F32))
    err = np.abs(first[small] + second * 2.0 ** -up - p[small])
    assert np.all(err <= 2.0 ** (-11 * terms) * p[small])
