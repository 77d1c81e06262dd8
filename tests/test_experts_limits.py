"""Limits of the routing, expert product and combine calls that follow from their launches and counters; only refusals
are called."""

import ctypes

import pytest

from test_experts_abi import experts, product, routing
from test_layer_abi import ENULL, ESHAPE, lib  # noqa: F401


@pytest.mark.parametrize("topk", range(1, 33))
def test_pairs_of_a_workgroup_are_counted_in_16_bits(lib, topk):   # noqa: F811
    """The workspace holds two bytes an expert (here 8) and workgroup; b workgroups of t tokens each take more than
    (b - 1) t of them."""
    for tokens in ((1 << 24) // topk, (1 << 24) // topk - 1, (1 << 23) // topk, 300000 // topk):
        blocks = lib.bitnet_route_workspace_bytes(tokens, topk, 8) // 16
        assert 2 <= blocks <= 513
        assert (tokens - 1) // (blocks - 1) * topk <= 65535


def test_products_beyond_a_launch(lib):   # noqa: F811
    """More than 2^24 - 9 workgroups of 32 rows and 256 outputs (128 with gate and up), and more outputs than 2^31 - 32."""
    def dense(rows, n, up):
        args = {} if up else dict(up=None, up_scale=None, up_bias=None)
        return lib.bitnet_ternary_linear_act(ctypes.byref(product(rows=rows, N=n, K=64, **args)), None)
    most = 2 ** 24 - 9
    assert dense(1, 2 ** 31 - 31, False) == ESHAPE
    assert dense(33, 2 ** 31 - 32, False) == ESHAPE
    assert dense(1, most * 128 + 1, True) == ESHAPE
    assert dense(32 * most + 1, 1, False) == ESHAPE and dense(1 << 30, 40, False) == ESHAPE
    assert dense(32 * (most // 2) + 1, 257, False) == ESHAPE and dense(32 * (most // 2) + 1, 129, True) == ESHAPE

    def grouped(slots, experts_, n):
        r = routing(tokens=slots, topk=1, experts=experts_)
        return experts(lib, r, product(rows=slots, N=n, K=64, up=None, up_scale=None, up_bias=None), 1)
    assert grouped(32 * (most - 1000 + 1), 1000, 1) == ESHAPE
    assert grouped(40, 1000, 256 * (most // 41) + 1) == ESHAPE


@pytest.mark.parametrize("k", [192, 320, 704, 4160, 131008, 128, 131072])
def test_weights_of_a_product_are_below_2_38(lib, k):   # noqa: F811
    """The largest N with N * K < 2^38 is no wrong size (the call without a matrix gets as far as its addresses),
    the next is."""
    n = (2 ** 38 - 1) // k

    def status(n):
        p = product(rows=1, N=n, K=k, w=None, up=None, up_scale=None, up_bias=None)
        return lib.bitnet_ternary_linear_act(ctypes.byref(p), None)
    assert status(min(n, 2 ** 31 - 32)) == ENULL and status(n + 1) == ESHAPE
