"""Refusals of the routing, expert product and combine calls: the C ABI rejects bad arguments before
any HIP call, the binding rejects bad tensors before the C call."""

import ctypes

import pytest
import torch

from ternary_weight_linear_bit_amd import _native as N

from test_layer_abi import (A, EALIGN, EDTYPE, ENULL, ESHAPE, EWS, OK, cpu, lib, z)  # noqa: F401

BIG = 1 << 40


def routing(**kw):
    f = dict(expert=A, weight=A, offset=A, pair=A, slot=A, tokens=5, topk=2, experts=8)
    f.update(kw)
    return N.BitnetRouting(*f.values())


def product(**kw):
    f = dict(w=A, up=A, w_scale=A, up_scale=A, bias=A, up_bias=A, x_q=A, x_scale=A, residual=None, y=A,
             rows=5, N=100, K=192, act=1, y_dtype=0)
    f.update(kw)
    return N.BitnetProduct(*f.values())


def route(lib, r, logits=A, dtype=0, stride=8, score=0, scale=1.0, ws=A, ws_bytes=BIG):   # noqa: F811
    return lib.bitnet_route(ctypes.byref(r), logits, dtype, stride, score, scale, ws, ws_bytes, None)


def experts(lib, r, p, by_slot=0):   # noqa: F811
    return lib.bitnet_expert_linear(ctypes.byref(r), ctypes.byref(p), by_slot, None)


def combine(lib, r, y=A, y_dtype=0, k=40, residual=A, out=A, out_dtype=0):   # noqa: F811
    return lib.bitnet_combine(ctypes.byref(r), y, y_dtype, k, residual, out, out_dtype, None)


SIZES = [dict(tokens=-1), dict(topk=0), dict(topk=33), dict(experts=0), dict(experts=1025),
         dict(tokens=(1 << 29) + 1), dict(tokens=1 << 62)]


@pytest.mark.parametrize("bad", SIZES)
def test_sizes_of_a_routing(lib, bad):   # noqa: F811
    r = routing(**bad)
    assert route(lib, r) == ESHAPE and route(lib, r, logits=None) == ESHAPE
    assert experts(lib, r, product(rows=max(r.tokens, 0))) == ESHAPE and combine(lib, r) == ESHAPE
    assert lib.bitnet_route_workspace_bytes(r.tokens, r.topk, r.experts) == 0


@pytest.mark.parametrize("rbad,bad,want", [
    ({}, dict(dtype=2), EDTYPE), ({}, dict(stride=7), ESHAPE), ({}, dict(score=3), ESHAPE),
    ({}, dict(score=-1), ESHAPE), ({}, dict(scale=float("nan")), ESHAPE), ({}, dict(scale=float("inf")), ESHAPE),
    (dict(expert=None), {}, ENULL), (dict(weight=None), {}, ENULL), (dict(offset=None), {}, ENULL),
    (dict(pair=None), {}, ENULL), (dict(slot=None), {}, ENULL), (dict(pair=A + 2), {}, EALIGN),
    (dict(offset=A + 1), {}, EALIGN), ({}, dict(logits=A + 2), EALIGN), ({}, dict(dtype=1, logits=A + 1), EALIGN)])
def test_route_refusals(lib, rbad, bad, want):   # noqa: F811
    assert route(lib, routing(**rbad), **bad) == want


def test_route_workspace(lib):   # noqa: F811
    big = routing(tokens=1 << 24, topk=2)
    assert route(lib, big) == ESHAPE and lib.bitnet_route_workspace_bytes(1 << 24, 2, 8) == 0
    assert lib.bitnet_route_workspace_bytes(1 << 23, 2, 8) > 0
    r = routing(tokens=100000)
    need = lib.bitnet_route_workspace_bytes(100000, 2, 8)
    assert need > 0 and lib.bitnet_route_workspace_bytes(0, 2, 8) == 0
    assert route(lib, r, ws=None) == EWS and route(lib, r, ws_bytes=need - 1) == EWS
    assert route(lib, r, ws=A + 8, ws_bytes=need) == EALIGN


BAD_PRODUCT = [
    (dict(y_dtype=2), EDTYPE), (dict(N=-1), ESHAPE), (dict(K=0), ESHAPE), (dict(K=32), ESHAPE), (dict(K=100), ESHAPE),
    (dict(K=131136), ESHAPE), (dict(N=1 << 31), ESHAPE), (dict(N=1 << 37), ESHAPE), (dict(act=4), ESHAPE),
    (dict(act=-1), ESHAPE), (dict(up=None), ESHAPE), (dict(up=None, up_scale=None), ESHAPE),
    (dict(up_scale=None), ENULL), (dict(w=None), ENULL), (dict(w_scale=None), ENULL), (dict(x_q=None), ENULL),
    (dict(x_scale=None), ENULL), (dict(y=None), ENULL), (dict(w=A + 8), EALIGN), (dict(up=A + 8), EALIGN),
    (dict(x_q=A + 4), EALIGN), (dict(y=A + 2), EALIGN), (dict(y_dtype=1, y=A + 1), EALIGN), (dict(bias=A + 2), EALIGN),
    (dict(up_bias=A + 2), EALIGN), (dict(w_scale=A + 2), EALIGN), (dict(up_scale=A + 1), EALIGN), (dict(x_scale=A + 2), EALIGN)]


@pytest.mark.parametrize("bad,want", BAD_PRODUCT + [(dict(rows=-1), ESHAPE), (dict(rows=(1 << 30) + 1), ESHAPE),
                                                    (dict(residual=A + 2), EALIGN)])
def test_product_refusals(lib, bad, want):   # noqa: F811
    assert lib.bitnet_ternary_linear_act(ctypes.byref(product(**bad)), None) == want


@pytest.mark.parametrize("bad,want", BAD_PRODUCT + [(dict(rows=4), ESHAPE), (dict(rows=10), ESHAPE),
                                                    (dict(residual=A), ESHAPE)])
def test_expert_refusals(lib, bad, want):   # noqa: F811
    assert experts(lib, routing(), product(**bad)) == want


def test_expert_routing_refusals(lib):   # noqa: F811
    p = product()
    assert experts(lib, routing(offset=None), p) == ENULL and experts(lib, routing(pair=None), p) == ENULL
    assert experts(lib, routing(offset=A + 2), p) == EALIGN and experts(lib, routing(), p, 2) == ESHAPE
    assert experts(lib, routing(), product(rows=5), 1) == ESHAPE             # by slot: 10 rows
    # gathered rows lie within 2^31 bytes
    assert experts(lib, routing(tokens=(1 << 24) + 1, topk=1), product(rows=(1 << 24) + 1, K=128)) == ESHAPE
    # a grid that the runtime cannot count
    huge = product(rows=1 << 30, N=1 << 24, K=64)
    assert lib.bitnet_ternary_linear_act(ctypes.byref(huge), None) == ESHAPE
    assert experts(lib, routing(tokens=1 << 30, topk=1), product(rows=1 << 30, N=1 << 24, K=64), 1) == ESHAPE
    assert lib.bitnet_ternary_linear_act(None, None) == ENULL
    assert lib.bitnet_expert_linear(None, ctypes.byref(p), 0, None) == ENULL
    assert lib.bitnet_expert_linear(ctypes.byref(routing()), None, 0, None) == ENULL


@pytest.mark.parametrize("rbad,bad,want", [
    ({}, dict(y_dtype=2), EDTYPE), ({}, dict(out_dtype=-1), EDTYPE), ({}, dict(k=-1), ESHAPE), ({}, dict(k=(1 << 23) + 1), ESHAPE),
    (dict(weight=None), {}, ENULL), (dict(slot=None), {}, ENULL), ({}, dict(y=None), ENULL), ({}, dict(out=None), ENULL),
    (dict(slot=A + 2), {}, EALIGN), ({}, dict(y=A + 2), EALIGN), ({}, dict(residual=A + 1), EALIGN),
    ({}, dict(out_dtype=1, out=A + 1), EALIGN)])
def test_combine_refusals(lib, rbad, bad, want):   # noqa: F811
    assert combine(lib, routing(**rbad), **bad) == want


def test_nothing_to_do(lib):   # noqa: F811
    none = routing(tokens=0, expert=None, weight=None, offset=None, pair=None, slot=None)
    assert experts(lib, none, product(rows=0, w=None, x_q=None, y=None)) == OK
    assert experts(lib, routing(), product(N=0, w=None, y=None)) == OK
    assert lib.bitnet_ternary_linear_act(ctypes.byref(product(rows=0, y=None)), None) == OK
    assert combine(lib, none, y=None, out=None) == OK and combine(lib, routing(), k=0, y=None, out=None) == OK
    assert lib.bitnet_route(None, A, 0, 8, 0, 1.0, A, BIG, None) == ENULL
    assert lib.bitnet_combine(None, A, 0, 8, A, A, 0, None) == ENULL


def test_packed_struct_matches_the_header():
    assert N._PRODUCT.size == ctypes.sizeof(N.BitnetProduct)
    v = tuple(range(1, 16))
    assert N._PRODUCT.pack(*v) == bytes(N.BitnetProduct(*v))


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------

I32, I8, U8 = torch.int32, torch.int8, torch.uint8


def a_routing(n, tokens=3, topk=2, experts=4):
    return n.Routing(z(tokens, topk, dtype=I32), z(tokens, topk), z(experts + 1, dtype=I32),
                     z(tokens * topk, dtype=I32), z(tokens, topk, dtype=I32))


def some_experts(n, e=4, rows=40, k=192):
    return n.TernaryExperts(z(e, *n.prefill_layout_shape(rows, k), dtype=U8), z(e), rows, k)


def test_binding_rejects_bad_handles(cpu):   # noqa: F811
    ok = (z(3, 2, dtype=I32), z(3, 2), z(5, dtype=I32), z(6, dtype=I32), z(3, 2, dtype=I32))
    cpu.Routing(*ok)
    for i, bad in ((0, z(3, 2)), (0, z(6, dtype=I32)), (1, z(3, 1)), (1, z(3, 2).double()), (2, z(1, dtype=I32)),
                   (2, z(5)), (3, z(5, dtype=I32)), (4, z(2, 3, dtype=I32)), (0, z(3, 0, dtype=I32))):
        with pytest.raises(ValueError):
            cpu.Routing(*ok[:i], bad, *ok[i + 1:])
    w = z(4, *cpu.prefill_layout_shape(40, 192), dtype=U8)
    for args in ((w, z(3), 40, 192), (w, z(4), 65, 192), (w, z(4), 40, 300), (w.float(), z(4), 40, 192),
                 (w, z(4).double(), 40, 192), (w, z(4, 1), 40, 192)):
        with pytest.raises(ValueError):
            cpu.TernaryExperts(*args)
    with pytest.raises(ValueError):
        cpu.TernaryExperts.from_packed(z(40, 48, dtype=U8), z(1))
    r = a_routing(cpu)
    with pytest.raises(AttributeError, match="fixed"):
        r.topk = 3


@pytest.mark.parametrize("bad", [
    dict(logits=z(3, 5)), dict(logits=z(2, 4)), dict(logits=z(3, 4).double()), dict(logits=z(4, 3).t()),
    dict(logits=z(1, 4).expand(3, 4)), dict(logits=z(3, 4), score="max"), dict(logits=z(12))])
def test_binding_rejects_bad_logits(cpu, bad):   # noqa: F811
    with pytest.raises(ValueError):
        cpu.bitnet_route(a_routing(cpu), **bad)


@pytest.mark.parametrize("bad", [
    dict(x_q=z(6, 192, dtype=I8)), dict(x_q=z(3, 128, dtype=I8)), dict(x_q=z(3, 192)), dict(x_scale=z(2)),
    dict(x_scale=z(3).double()), dict(bias=z(40)), dict(bias=z(4, 41)), dict(up_bias=z(4, 40)), dict(act="relu"),
    dict(y=z(3, 40)), dict(y=z(6, 40).double()), dict(y=z(6, 40), y_dtype=torch.bfloat16), dict(slots=True)])
def test_binding_rejects_bad_products(cpu, bad):   # noqa: F811
    args = dict(x_q=z(3, 192, dtype=I8), x_scale=z(3))
    args.update(bad)
    with pytest.raises(ValueError):
        cpu.bitnet_expert_linear(a_routing(cpu), some_experts(cpu), **args)
    with pytest.raises(ValueError):
        cpu.bitnet_expert_linear(a_routing(cpu, experts=5), some_experts(cpu), z(3, 192, dtype=I8), z(3))
    with pytest.raises(ValueError):
        cpu.bitnet_expert_linear(a_routing(cpu), some_experts(cpu), z(3, 192, dtype=I8), z(3), up=some_experts(cpu, rows=41))


@pytest.mark.parametrize("bad", [
    dict(w_prefill=z(1, 2048, dtype=U8)), dict(n=65), dict(w_scale=z(1).double()), dict(x_q=z(3, 128, dtype=I8)),
    dict(x_q=z(192, dtype=I8)), dict(bias=z(1, 40)), dict(residual=z(3, 41)), dict(residual=z(3, 40), y_dtype=torch.bfloat16),
    dict(up=(z(2, 1024, dtype=U8), z(1))), dict(y=z(4, 40)), dict(act=None)])
def test_binding_rejects_bad_dense_products(cpu, bad):   # noqa: F811
    args = dict(w_prefill=z(2, 2048, dtype=U8), w_scale=z(1), n=40, x_q=z(3, 192, dtype=I8), x_scale=z(3))
    args.update(bad)
    with pytest.raises(ValueError):
        cpu.bitnet_ternary_linear_act(**args)


@pytest.mark.parametrize("bad", [
    dict(y=z(5, 8)), dict(y=z(48)), dict(y=z(6, 8).double()), dict(out=z(3, 9)), dict(out=z(3, 8), out_dtype=torch.bfloat16),
    dict(residual=z(6, 8)), dict(residual=z(3, 8), out_dtype=torch.bfloat16), dict(out=z(3, 8).half())])
def test_binding_rejects_bad_combinations(cpu, bad):   # noqa: F811
    args = dict(y=z(6, 8))
    args.update(bad)
    with pytest.raises(ValueError):
        cpu.bitnet_combine(a_routing(cpu), **args)
