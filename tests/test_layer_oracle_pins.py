"""The layer oracle against values that do not come from it: hand-worked pages,
complex multiplication, Python's fractions, a softmax by hand, closed forms."""

import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import bitnet_oracle as O
from oracle import layer_oracle as L

F32 = np.float32


def test_rotation_is_complex_multiplication():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 10)).astype(F32)
    ang = rng.uniform(0, 6, 4)
    c, s = np.cos(ang).astype(F32), np.sin(ang).astype(F32)
    for inter in (False, True):
        y = L.rotate(x, c, s, inter)
        ia = np.arange(4) * 2 if inter else np.arange(4)
        ib = ia + (1 if inter else 4)
        z = (x[:, ia].astype(np.float64) + 1j * x[:, ib]) * (c.astype(np.float64) + 1j * s)
        # three roundings, each at most 2^-24 of a term of at most |x| 2
        np.testing.assert_allclose(y[:, ia], z.real, atol=3 * 2.0 ** -24 * 8)
        np.testing.assert_allclose(y[:, ib], z.imag, atol=3 * 2.0 ** -24 * 8)
        np.testing.assert_array_equal(y[:, 8:], x[:, 8:])      # the rest passes through


def test_rotation_rounds_each_product():
    # a c = 1 + 2^-23 + 2^-46 rounds to 1 + 2^-23; a fused form would keep the last term
    a, c = F32(1 + 2.0 ** -23), F32(1 + 2.0 ** -23)
    b, s = F32(1.0), F32(1 + 2.0 ** -22)
    got = L.rotate(np.array([a, b], F32), [c], [s], True)[0]
    assert got == F32(0.0)
    assert float(a) * float(c) - float(b) * float(s) != 0.0


def test_append_page_by_hand():
    # 127 * 0.5 / 0.5: the page begins, need = 63.5 / 127 = 0.5
    codes = np.full((4, 2), 99, np.int8)
    d = L.append_page(codes, F32(77.0), np.array([[63.5, -1.25], [0.25, 0.75]], F32), 0)
    assert d == F32(0.5)
    # -2.5 -> -2 and 0.5 -> 0, 1.5 -> 2: ties to even; slots behind keep their bytes
    np.testing.assert_array_equal(codes, [[127, -2], [0, 2], [99, 99], [99, 99]])
    # a smaller row leaves the scale: 10 / 0.5
    assert L.append_page(codes, d, np.array([[10.0, 0.0]], F32), 2) == F32(0.5)
    np.testing.assert_array_equal(codes, [[127, -2], [0, 2], [20, 0], [99, 99]])
    # 127 doubles the scale; 127 / 2 = 63.5 -> 64, -2 / 2 = -1, 2 / 2 = 1, 20 / 2 = 10
    assert L.append_page(codes, F32(0.5), np.array([[127.0, 3.0]], F32), 3) == F32(1.0)
    np.testing.assert_array_equal(codes, [[64, -1], [0, 1], [10, 0], [127, 3]])


def test_scale_floor():
    codes = np.zeros((2, 2), np.int8)
    d = L.append_page(codes, F32(0), np.zeros((1, 2), F32), 0)
    want = Fraction(float(F32(1e-5))) / 127
    assert abs(Fraction(float(d)) - want) <= want * Fraction(1, 2 ** 24)
    np.testing.assert_array_equal(codes, 0)


def test_append_places_rows():
    """7 rows of one sequence behind 3 tokens, pages of 4 out of order, one page missing."""
    P, D = 4, 2
    k = np.full((5, 1, P, D), 50, np.int8)
    v = np.full((5, 1, D, P), 51, np.int8)
    ks, vs = np.full((5, 1), 1.0, F32), np.full((5, 1), 1.0, F32)
    rows = np.arange(1, 8, dtype=F32)[:, None, None] * np.ones((7, 1, D), F32)
    table = np.array([[3, 9, 1]], np.int32)               # page 9 does not exist
    k2, v2, ks2, vs2, _ = L.kv_append(k, v, ks, vs, table, np.array([0, 7]), np.array([10]), rows,
                                      rows)
    assert k2[3, 0, 3, 0] == 1 and v2[3, 0, 1, 3] == 1        # position 3: scale 1 stays
    np.testing.assert_array_equal(k2[3, 0, :3], 50)
    # positions 8, 9 (rows 6 and 7) begin page 1: scale 7/127
    assert ks2[1, 0] == F32(7) / F32(127)
    assert k2[1, 0, 1, 0] == 127 and k2[1, 0, 0, 0] == round(6 * 127 / 7)
    np.testing.assert_array_equal(v2[1, 0, :, 1], 127)
    for pid in (0, 2, 4):
        np.testing.assert_array_equal(k2[pid], k[pid])
        assert ks2[pid] == ks[pid]


def test_attention_by_hand():
    """Two keys with logits ln 3 apart weigh 3/4 and 1/4."""
    k = np.zeros((1, 1, 4, 2), np.int8)
    k[0, 0, 0] = [1, 0]
    v = np.zeros((1, 1, 2, 4), np.int8)
    v[0, 0, :, 0], v[0, 0, :, 1] = [8, 0], [0, 8]
    v[0, 0, :, 2] = 127                                       # not visible
    one, two = np.ones((1, 1), F32), np.full((1, 1), 2.0, F32)
    q = np.array([[[math.log(3.0), 5.0]]])
    out, lse = L.attention(k, v, one, two, np.array([[0]]), np.array([0, 1]), np.array([2]), q, 1.0)
    np.testing.assert_allclose(out[0, 0], [12.0, 4.0], rtol=1e-12)
    np.testing.assert_allclose(lse[0, 0], math.log(4.0), rtol=1e-12)
    # a window of one key: the row's own
    out, lse = L.attention(k, v, one, two, np.array([[0]]), np.array([0, 1]), np.array([2]), q, 1.0,
                           window=1)
    np.testing.assert_allclose(out[0, 0], [0.0, 16.0])
    np.testing.assert_allclose(lse[0, 0], 0.0, atol=1e-15)


def test_attention_is_causal_and_grouped():
    """Row i of several sees exactly the keys up to itself; constant values come back."""
    rng = np.random.default_rng(3)
    k = rng.integers(-127, 128, (3, 2, 16, 16)).astype(np.int8)
    v = np.broadcast_to(np.arange(1, 17, dtype=np.int8), (3, 2, 16, 16)).copy()   # v[d, slot] = slot + 1
    one = np.ones((3, 2), F32)
    q = np.zeros((3, 4, 16))                                  # equal weights
    out, lse = L.attention(k, v, one, one, np.array([[2]]), np.array([0, 3]), np.array([5]), q, 1.0)
    for i, n in enumerate((3, 4, 5)):
        np.testing.assert_allclose(out[i], np.mean(np.arange(1, n + 1)))
        np.testing.assert_allclose(lse[i], math.log(n))
    # more rows than tokens: the first see nothing
    out, lse = L.attention(k, v, one, one, np.array([[2]]), np.array([0, 3]), np.array([1]), q, 1.0)
    np.testing.assert_array_equal(out[:2], 0.0)
    assert np.all(np.isneginf(lse[:2])) and np.all(lse[2] == 0.0)


def test_residual_by_hand():
    # y = (3, 4, 0, 0): mean of squares 25/4, r = 0.4 (eps 0) -> z = (1.2, 1.6, 0, 0)
    y = np.array([[3, 4, 0, 0]], F32)
    h = np.array([[10, 20, 30, 40]], F32)
    w = np.array([1, 2, 1, 1], F32)
    h2, u, xq, d = L.residual_norm(y, h, post_weight=w, gate=np.array([2, 0.5, 1, 1], F32), scale=0.5,
                                   eps=0.0)
    r = F32(1.0 / math.sqrt(6.25))
    np.testing.assert_array_equal(h2, [[10 + F32(3) * r, 20 + F32(F32(4) * r) * F32(2) * F32(0.25), 30, 40]])
    np.testing.assert_array_equal(u, h2)
    assert xq[0, 3] == 127 and d[0] == F32(40) / F32(127)


def test_residual_stream_is_rounded_before_the_norm():
    """With a bf16 stream the next norm sees the stored values."""
    h = np.array([[256.0, 0.0]], F32)
    y = np.array([[0.5, 1.0]], F32)                            # 256.5 is not a bf16 value
    h2, u, _, _ = L.residual_norm(y, h, h_bf16=True, pre_weight=np.ones(2, F32))
    assert h2[0, 0] == 256.0
    _, u32, _, _ = L.residual_norm(y, h, h_bf16=False, pre_weight=np.ones(2, F32))
    assert not np.array_equal(u, u32)


def test_residual_without_norms_is_the_quantiser():
    rng = np.random.default_rng(5)
    y, h = rng.standard_normal((2, 3, 40)).astype(F32)
    h2, u, xq, d = L.residual_norm(y, h)
    np.testing.assert_array_equal(h2, h + y)
    want_q, want_d = O.quantize_acts(h + y)
    np.testing.assert_array_equal(xq, want_q)
    np.testing.assert_array_equal(d, want_d)


@pytest.mark.parametrize("plant", ["old_scale_kept", "need_without_floor", "per_row_scale"])
def test_planted_scale_mistakes_are_seen(monkeypatch, plant):
    """A wrong page scale fails the hand-worked page or the floor."""
    def wrong(x, old):
        need = F32(np.abs(x).max()) / O.QB
        if plant == "old_scale_kept":
            return F32(max(need, O.EPS / O.QB)) if old is None else F32(old)
        if plant == "need_without_floor":
            return max(need, F32(1e-20)) if old is None else max(F32(old), need)
        need = F32(np.abs(x[-1]).max()) / O.QB                # the last row's maximum only
        return max(need, F32(O.EPS / O.QB)) if old is None else max(F32(old), need)
    monkeypatch.setattr(L, "page_scale", wrong)
    with pytest.raises(AssertionError):
        test_append_page_by_hand()
        test_scale_floor()
