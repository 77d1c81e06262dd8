"""The experts' oracle against values that do not come from it: choices and plans by hand,
softmax identities, Python's fractions, the dense oracle."""

import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import bitnet_oracle as O
from oracle import experts_oracle as E

F32 = np.float32
INF = float("inf")


def test_choice_by_hand():
    x = np.array([[1, 3, 3, 2], [-INF, 5, float("nan"), -INF], [0.0, -0.0, INF, INF], [-INF] * 4])
    np.testing.assert_array_equal(E.choose(x, 3), [[1, 2, 3], [1, -1, -1], [2, 3, 0], [-1, -1, -1]])


def test_weights_by_hand():
    x = np.log(np.array([[1.0, 2.0, 5.0, 8.0]]))
    e = E.choose(x, 2)
    np.testing.assert_array_equal(e, [[3, 2]])
    np.testing.assert_allclose(E.weigh(x, e, "softmax", 2.0), [[1.0, 10 / 16]], rtol=1e-14)
    np.testing.assert_allclose(E.weigh(x, e, "chosen", 1.0), [[8 / 13, 5 / 13]], rtol=1e-14)
    np.testing.assert_allclose(E.weigh(x, e, "sigmoid", 1.0), [[8 / 9, 5 / 6]], rtol=1e-14)
    y = np.array([[INF, 0.0, INF], [2.0, -INF, -INF], [-INF] * 3])
    e = E.choose(y, 2)
    np.testing.assert_array_equal(E.weigh(y, e, "softmax", 1.0), [[0.5, 0.5], [1, 0], [0, 0]])
    np.testing.assert_array_equal(E.weigh(y, e, "sigmoid", 1.0)[0], [1, 1])


def test_plan_by_hand():
    offset, pair, slot = E.plan([[2, 0], [-1, 2], [0, 7]], 3)
    np.testing.assert_array_equal(offset, [0, 2, 2, 4])
    np.testing.assert_array_equal(pair, [1, 4, 0, 3, -1, -1])
    np.testing.assert_array_equal(slot, [[2, 0], [-1, 3], [1, -1]])


@pytest.mark.parametrize("seed", range(3))
def test_plan_inverts(seed):
    rng = np.random.default_rng(seed)
    e = rng.integers(-1, 6, (40, 3))
    offset, pair, slot = E.plan(e, 6)
    flat = e.reshape(-1)
    assert offset[-1] == (flat >= 0).sum()
    for x in range(6):
        mine = pair[offset[x]:offset[x + 1]]
        assert (flat[mine] == x).all() and (np.diff(mine) > 0).all()
        np.testing.assert_array_equal(slot.reshape(-1)[mine], np.arange(offset[x], offset[x + 1]))


def test_product_is_the_dense_layer():
    rng = np.random.default_rng(5)
    q = rng.integers(-1, 2, (7, 64))
    x, d = rng.integers(-128, 128, (5, 64)).astype(np.int8), rng.random(5).astype(F32)
    acc, y = O.ternary_linear(O.pack_codes(q.astype(np.int8)), F32(0.3), x, d)[:2]
    got, tol = E.product(q, F32(0.3), x, d)
    assert tol is None
    np.testing.assert_array_equal(E.accumulate(q, x), acc)
    np.testing.assert_array_equal(got, y)


def rn(x):
    return F32(float(x))        # fractions with at most 53 bits here: one rounding


def test_epilogue_rounds_each_step():
    q, x = np.array([[1, -1, 0, 1]]), np.array([[100, 27, 5, 3]], np.int8)
    up = (np.array([[0, 1, 1, 0]]), F32(0.7), np.array([0.125], F32))
    g, d, b, res = F32(0.1), np.array([0.3], F32), np.array([0.01], F32), np.array([[3.3]], F32)
    v = rn(Fraction(float(rn(76 * Fraction(float(rn(Fraction(float(g)) * Fraction(float(d[0])))))))) + Fraction(float(b[0])))
    a = rn(Fraction(float(v)) ** 2)
    u = rn(Fraction(float(rn(32 * Fraction(float(rn(Fraction(float(up[1])) * Fraction(float(d[0])))))))) + Fraction(1, 8))
    want = rn(Fraction(float(rn(Fraction(float(a)) * Fraction(float(u))))) + Fraction(float(res[0, 0])))
    got, tol = E.product(q, g, x, d, b, "relu2", up, res)
    assert tol is None and got[0, 0] == want
    assert E.product(-q, g, x, d, None, "relu2")[0][0, 0] == 0.0


def test_activations():
    v = np.array([-3.0, -0.5, 0.0, 0.5, 3.0, -90.0, 90.0], F32)
    s, g = E.activate(v, "silu"), E.activate(v, "gelu")
    for z, a, b in zip(v.astype(float), s, g):
        assert math.isclose(a, z / (1 + math.exp(-z)), rel_tol=1e-14, abs_tol=0)
        # the distribution function by its integral from 0, in small steps
        n = 20000
        t = np.linspace(0, min(max(z, -12), 12), n + 1)
        f = np.exp(-t * t / 2) / math.sqrt(2 * math.pi)
        area = 0.5 + float(((f[1:] + f[:-1]) / 2 * np.diff(t)).sum())
        assert abs(b - z * area) <= 1e-6 * abs(z) + 1e-300
    np.testing.assert_array_equal(E.activate(v, "none"), v)


def test_combine_by_hand():
    y = np.array([[1, 2], [10, 20], [100, 200]], F32)
    w = np.array([[0.5, 2.0], [1.0, 3.0]], F32)
    slot = np.array([[2, 0], [-1, 5]])
    np.testing.assert_array_equal(E.combine(w, slot, y), [[52, 104], [0, 0]])
    np.testing.assert_array_equal(E.combine(w, slot, y, np.ones((2, 2))), [[53, 105], [1, 1]])
    # products and sums round by themselves: 1 + 2^-24 is 1, a fused form would give 1 + 2^-23
    a = F32(1 + 2.0 ** -12)
    one = E.combine(np.array([[a]], F32), np.array([[0]]), np.array([[a]], F32), np.array([[F32(2.0 ** -24)]]))
    assert one[0, 0] == F32(F32(float(a) ** 2) + F32(2.0 ** -24))
