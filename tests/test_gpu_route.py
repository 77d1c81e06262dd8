"""bitnet_route and bitnet_combine on the GPU against the oracle: indices and combinations bit for
bit, weights within bounds derived from fp32."""

import numpy as np
import pytest
import torch

from oracle import experts_oracle as E
from ternary_weight_linear_bit_amd import _native as N

from experts_util import F32, TORCH, assign, dev, host, routing, same, typed
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.lib()


def check(r, x, topk, score="softmax", scale=1.0):
    """The routing's arrays against the oracle on fp32 logits x."""
    want = E.choose(x, topk)
    np.testing.assert_array_equal(host(r.expert), want)
    for got, plan in zip((r.offset, r.pair, r.slot), E.plan(want, x.shape[1])):
        np.testing.assert_array_equal(host(got), plan)
    w = E.weigh(x, want, score, scale)
    # differences of fp32 logits are rounded to 2^-24 of up to twice the largest, which moves e^(x - m)
    # by as much of itself times that size; beside it exp, the sum over the experts, the quotient and the scale:
    # a few roundings each, the sum's in log2 E + E / 64 steps
    n = x.shape[1]
    top = np.where(np.isfinite(x), np.abs(x), 0).max(-1, keepdims=True)
    tol = (2 * top + n / 64 + 32) * 2.0 ** -24
    got = host(r.weight).astype(np.float64)
    assert np.all(np.abs(got - w) <= tol * np.abs(w) + 1e-37)
    np.testing.assert_array_equal(got[want < 0], 0)


def logits(tokens, experts, seed, dt, ties=False):
    rng = np.random.default_rng(seed)
    x = 2 * rng.standard_normal((tokens, experts))
    return typed(np.round(x) if ties else x, dt)


@pytest.mark.parametrize("score", ["softmax", "chosen", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,topk,dt", [
    (1, 1, 1, "f32"), (1, 8, 2, "bf16"), (3, 63, 32, "f32"), (64, 64, 6, "bf16"), (65, 65, 1, "f32"), (129, 128, 8, "bf16"),
    (200, 129, 3, "f32"), (37, 256, 8, "f32"), (300, 257, 7, "bf16"), (33, 512, 5, "f32"), (40, 513, 9, "bf16"), (17, 1024, 32, "f32"),
    (1500, 16, 4, "f32"), (5, 2, 5, "f32"), (700, 1000, 3, "bf16"), (17000, 40, 32, "bf16")])
def test_route(tokens, experts, topk, dt, score):
    t, x = logits(tokens, experts, tokens + experts, dt)
    r = N.bitnet_route(N.Routing.empty(tokens, topk, experts, DEV), t, score, 1.25)
    check(r, x, topk, score, 1.25)


@pytest.mark.parametrize("experts", [8, 60, 250, 1000])
def test_ties_take_the_lowest_index(experts):
    t, x = logits(150, experts, experts, "f32", ties=True)
    t[0], x[0] = 0.0, 0.0
    t[1, ::2], x[1, ::2] = -0.0, -0.0                      # equal to 0
    t[1, 1::2], x[1, 1::2] = 0.0, 0.0
    check(N.bitnet_route(N.Routing.empty(150, 5, experts, DEV), t), x, 5)


@pytest.mark.parametrize("score", ["softmax", "chosen", "sigmoid"])
def test_masked_logits(score):
    _, x = logits(200, 40, 3, "f32")
    x = x.copy()
    x[:, 7:31] = -INF                    # experts switched off
    x[10] = -INF                         # a token without experts
    x[11, 1:] = -INF                     # with one
    x[12, 2:] = np.nan
    x[13] = np.nan
    x[14, 3] = INF
    x[15, [2, 5, 33]] = INF
    x[16] = np.finfo(F32).min            # the type's lowest value is a logit like others
    x[17, :] = -INF
    x[17, 4:9] = np.finfo(F32).min
    x[190:] = -INF                       # padding
    r = N.bitnet_route(N.Routing.empty(200, 6, 40, DEV), dev(x), score)
    want = E.choose(x, 6)
    np.testing.assert_array_equal(host(r.expert), want)
    for got, plan in zip((r.offset, r.pair, r.slot), E.plan(want, 40)):
        np.testing.assert_array_equal(host(got), plan)
    rows = np.r_[0:16, 18:200]           # (weights of finite and masked rows)
    rows = rows[rows != 16]
    w = E.weigh(x[rows], want[rows], score, 1.0)
    np.testing.assert_allclose(host(r.weight)[rows], w, rtol=64 * 2.0 ** -24, atol=0)
    # equal logits share the weight; sigmoid of the lowest value is 0
    equal = {"softmax": (1 / 40, 1 / 5), "chosen": (1 / 6, 1 / 5), "sigmoid": (0, 0)}[score]
    np.testing.assert_allclose(host(r.weight)[16], np.full(6, equal[0]), rtol=1e-6)
    np.testing.assert_allclose(host(r.weight)[17], [equal[1]] * 5 + [0], rtol=1e-6)


def test_rows_apart_and_unaligned():
    rng = np.random.default_rng(8)
    for dt, pad, at in (("f32", 13, 3), ("bf16", 7, 1), ("f32", 0, 0)):
        t, x = typed(rng.standard_normal((90, 50 + pad)), dt)
        check(N.bitnet_route(N.Routing.empty(90, 4, 50, DEV), t[:, at:at + 50]), x[:, at:at + 50], 4)


@pytest.mark.parametrize("tokens,topk,experts", [(1, 1, 1), (7, 3, 5), (512, 1, 3), (300, 7, 64), (171, 3, 1000), (4000, 8, 33),
                                                 (70001, 16, 300), (600000, 1, 5)])
def test_plan_of_given_experts(tokens, topk, experts):
    """Numbers outside the experts have no slot; the same expert may come twice; weights stay."""
    e = np.random.default_rng(tokens).integers(-3, experts + 3, (tokens, topk)).astype(np.int32)
    r = N.Routing.empty(tokens, topk, experts, DEV)
    r.expert.copy_(dev(e))
    r.weight.fill_(0.25)
    assert N.bitnet_route(r) is r
    np.testing.assert_array_equal(host(r.expert), e)
    assert (host(r.weight) == 0.25).all()
    inside = np.where((e >= 0) & (e < experts), e, -1)
    flat = inside.reshape(-1)
    order = np.argsort(np.where(flat < 0, experts, flat), kind="stable")
    count = np.bincount(flat[flat >= 0], minlength=experts)
    used = int(count.sum())
    np.testing.assert_array_equal(host(r.offset), np.r_[0, np.cumsum(count)])
    np.testing.assert_array_equal(host(r.pair), np.r_[order[:used], np.full(flat.size - used, -1)])
    slot = np.full(flat.size, -1)
    slot[order[:used]] = np.arange(used)
    np.testing.assert_array_equal(host(r.slot).reshape(-1), slot)


def test_no_tokens():
    r = N.Routing.empty(0, 2, 5, DEV)
    r.offset.fill_(9)
    N.bitnet_route(r, torch.empty((0, 5), device=DEV))
    assert (host(r.offset) == 0).all()
    r.offset.fill_(9)
    N.bitnet_route(r)
    assert (host(r.offset) == 0).all()


@pytest.mark.parametrize("tokens", [40, 3000])
def test_captured_route_follows_its_logits(tokens):
    """Two graphs with a workspace each, replayed with new contents and eager calls between."""
    outs, graphs = [], []
    t = torch.zeros((tokens, 24), device=DEV)
    for topk in (2, 5):
        r = N.Routing.empty(tokens, topk, 24, DEV)
        N.bitnet_route(r, t)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            N.bitnet_route(r, t)
        outs.append(r)
        graphs.append(g)
    for seed in range(4):
        x = np.random.default_rng(seed).standard_normal((tokens, 24)).astype(F32)
        t.copy_(dev(x))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for r, topk in zip(outs, (2, 5)):
            check(r, x, topk)
        N.bitnet_route(N.Routing.empty(tokens, 3, 24, DEV), t)
        torch.cuda.synchronize()


def test_another_stream():
    t, x = logits(500, 32, 4, "f32")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r = N.bitnet_route(N.Routing.empty(500, 4, 32, DEV), t, stream=s)
    s.synchronize()
    check(r, x, 4)
    with torch.cuda.stream(s):
        check(N.bitnet_route(N.Routing.empty(500, 4, 32, DEV), t, "chosen"), x, 4, "chosen")


# ---------------------------------------------------------------------------
# combination
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("yd,od", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("tokens,topk,k,residual,offset", [
    (1, 1, 1, False, 0), (1, 2, 2560, True, 0), (5, 3, 33, True, 0), (70, 8, 128, False, 0), (9, 32, 40, True, 0),
    (301, 2, 129, True, 1), (64, 6, 2560, True, 0), (33, 4, 1000, False, 3), (3, 2, 8200, True, 0)])
def test_combine(tokens, topk, k, residual, offset, yd, od):
    rng = np.random.default_rng(tokens + k)
    expert = rng.integers(-1, 9, (tokens, topk))
    r, (_, _, slot) = routing(expert, 9)

    def place(x, dt):
        t, f = typed(x, dt)
        flat = torch.zeros(t.numel() + offset, dtype=t.dtype, device=DEV)
        flat[offset:] = t.reshape(-1)
        return flat[offset:].view(t.shape), f
    y, yf = place(rng.standard_normal((tokens * topk, k)), yd)
    res, rf = place(3 * rng.standard_normal((tokens, k)), od) if residual else (None, None)
    want = E.combine(host(r.weight), slot, yf, rf)
    same(N.bitnet_combine(r, y, res, out_dtype=TORCH[od]), want, od)
    if residual:                                  # in place
        assert N.bitnet_combine(r, y, res, out=res) is res
        same(res, want, od)


def test_combine_of_many_tokens():
    """More tokens than workgroups in the first dimension: 65535 parts of a row leave 255 of them."""
    k, tokens = 65535 * 256 // 2, 3
    r, (_, _, slot) = routing([[0], [-1], [0]], 1)
    y = torch.zeros((tokens, k), dtype=torch.bfloat16, device=DEV)
    y[0], y[1] = 2.0, -4.0
    out = N.bitnet_combine(r, y)
    w = host(r.weight)
    for m, v in ((0, 2.0 * w[0, 0]), (1, 0.0), (2, -4.0 * w[2, 0])):
        assert bool((out[m] == torch.tensor(v, dtype=torch.float32).to(torch.bfloat16).to(DEV)).all())
    tokens = 200000
    r, (_, _, slot) = routing(np.zeros((tokens, 1), np.int32), 1)
    y, yf = typed(np.random.default_rng(2).standard_normal((tokens, 33)), "f32")
    same(N.bitnet_combine(r, y), (host(r.weight) * yf).astype(F32), "f32")


def test_combine_leaves_out_what_has_no_slot():
    r, _ = routing(assign([3, 2], 5, 2), 2)
    y, yf = typed(np.random.default_rng(1).standard_normal((10, 64)), "f32")
    y[5:] = float("nan")                          # behind the last slot: never read
    slot = np.array([[0, 1], [-1, -1], [10, 4], [1 << 30, -5], [2, 2]], np.int32)   # out of range, and one twice
    r.slot.copy_(dev(slot))
    same(N.bitnet_combine(r, y), E.combine(host(r.weight), slot, np.where(np.arange(10)[:, None] < 5, yf, 0)), "f32")


def test_empty_combinations():
    r = N.Routing.empty(0, 2, 3, DEV)
    assert N.bitnet_combine(r, torch.empty((0, 8), device=DEV)).shape == (0, 8)
    r, _ = routing(assign([1], 2, 1), 1)
    assert N.bitnet_combine(r, torch.empty((2, 0), device=DEV)).shape == (2, 0)
