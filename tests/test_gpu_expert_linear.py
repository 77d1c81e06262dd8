"""bitnet_expert_linear and bitnet_ternary_linear_act on the GPU against the oracle: bit for bit
without silu and gelu, within their stated bounds with them."""

import numpy as np
import pytest
import torch

from oracle import experts_oracle as E
from ternary_weight_linear_bit_amd import _native as N

from experts_util import F32, TORCH, acts, assign, close, dev, host, matrices, routing, same, typed
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.lib()


def compare(t, a, tol, dt):
    if tol is None:
        same(t, a, dt)
    else:
        close(t, a, tol, dt)


def run(counts, tokens, topk, n, k, act="none", gated=False, bias=False, slots=False, dt="f32", seed=0, expert=None,
        offset=0):
    """One call against the oracle, rows behind the last slot and around y looked at too."""
    print(f"counts={counts} tokens={tokens} topk={topk} N={n} K={k} {act} gated={gated} slots={slots} {dt}", flush=True)
    experts = len(counts)
    expert = assign(counts, tokens, topk, seed) if expert is None else expert
    r, (first, pair, _) = routing(expert, experts)
    pairs = tokens * topk
    xq, d = acts(pairs if slots else tokens, k, seed)
    rng = np.random.default_rng(seed + 77)
    mats = [matrices(experts, n, k, seed + 1 + i) for i in range(1 + gated)]
    b = [rng.standard_normal((experts, n)).astype(F32) if bias else None for _ in mats]
    buf = torch.full((pairs * n + 64,), 7.0, dtype=TORCH[dt], device=DEV)
    y = buf[32 + offset:32 + offset + pairs * n].view(pairs, n)
    got = N.bitnet_expert_linear(r, mats[0][2], dev(xq), dev(d), slots=slots, act=act, bias=None if not bias else dev(b[0]),
                                 up=mats[1][2] if gated else None, up_bias=dev(b[1]) if gated and bias else None, y=y)
    assert got is y
    for e in range(experts):
        s0, s1 = int(first[e]), int(first[e + 1])
        if s0 == s1:
            continue
        rows = np.arange(s0, s1) if slots else pair[s0:s1] // topk
        up = (mats[1][0][e], mats[1][1][e], b[1][e] if bias else None) if gated else None
        want = E.product(mats[0][0][e], mats[0][1][e], xq[rows], d[rows], b[0][e] if bias else None, act, up)
        compare(y[s0:s1], *want, dt)
    torch.cuda.synchronize()
    left = buf.float().cpu().numpy()
    assert (left[:32 + offset] == 7).all() and (left[32 + offset + pairs * n:] == 7).all()
    assert (y[int(first[-1]):].float().cpu().numpy() == 7).all()
    return y


# rows of each expert around the tiles' edges; every N and K is a different raggedness
COUNTS = [([1], 1, 1), ([0, 1, 0], 1, 1), ([1, 1], 1, 2), ([5, 0, 31, 32, 33], 60, 2), ([63, 0, 64, 65, 0, 1], 100, 2),
          ([127, 129, 128, 2], 200, 2), ([255, 0, 257, 256], 400, 2), ([0, 0, 600], 300, 2), ([1] * 70, 25, 3),
          ([0] * 64 + [3, 0, 2] + [0] * 61, 5, 1)]


@pytest.mark.parametrize("counts,tokens,topk", COUNTS)
@pytest.mark.parametrize("n,k", [(1, 64), (33, 192), (100, 128), (257, 320)])
def test_ragged(counts, tokens, topk, n, k):
    run(counts, tokens, topk, n, k, seed=len(counts))


@pytest.mark.parametrize("counts,tokens,topk", [COUNTS[1], COUNTS[3], COUNTS[6]])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("slots", [False, True])
@pytest.mark.parametrize("act", ["none", "relu2", "silu", "gelu"])
@pytest.mark.parametrize("gated,bias", [(False, False), (True, False), (True, True), (False, True)])
def test_epilogues(counts, tokens, topk, act, gated, bias, slots, dt):
    run(counts, tokens, topk, 90, 192, act, gated, bias, slots, dt, seed=3)


@pytest.mark.parametrize("n,k,dt", [(2560, 1152, "f32"), (864, 2560, "bf16"), (64, 14336, "bf16"), (40, 131072, "f32")])
def test_model_sizes(n, k, dt):
    run([70, 0, 3, 300], 190, 2, n, k, "relu2", True, False, False, dt, seed=5)
    run([2, 1], 3, 1, n, k, "none", False, True, True, dt, seed=6)


# wide enough for the kernels of many rows and each of their tiles, ragged in all directions
@pytest.mark.parametrize("counts,tokens,n", [([300], 150, 24001), ([150], 75, 24001), ([150], 80, 4001), ([40, 0, 33, 70], 72, 6016),
                                             ([257, 0, 384, 200], 421, 12008)])
@pytest.mark.parametrize("k,act,gated,bias,slots,dt", [
    (64, "none", False, False, False, "f32"), (192, "relu2", True, True, True, "bf16"), (128, "silu", False, True, False, "bf16"),
    (320, "none", False, True, True, "bf16"), (448, "gelu", True, False, False, "f32")])
def test_wide(counts, tokens, n, k, act, gated, bias, slots, dt):
    run(counts, tokens, 2, n, k, act, gated, bias, slots, dt, seed=n)


# the tiles that the sizes above do not reach: k steps shared by groups of waves, of which some have no
# step or a half one, and many slots under few columns
@pytest.mark.parametrize("counts,tokens,topk,n,k,act,gated,bias,slots,dt", [
    ([70, 33, 0, 90], 100, 2, 1600, 192, "relu2", False, False, False, "f32"),
    ([70, 33, 0, 90], 100, 2, 1601, 64, "none", False, True, True, "bf16"),
    ([70, 33, 0, 90], 100, 2, 1600, 192, "silu", True, True, False, "bf16"),
    ([70, 33, 0, 90], 100, 2, 1597, 704, "relu2", True, False, True, "f32"),
    ([70, 33, 0, 90], 100, 2, 795, 8256, "relu2", True, True, False, "bf16"),
    ([3, 0, 1], 2, 2, 70, 8256, "relu2", True, False, True, "f32"),
    ([436], 436, 1, 12008, 320, "relu2", True, True, False, "bf16"),
    ([10870], 10870, 1, 763, 576, "relu2", False, True, False, "bf16"),
    ([10880], 10880, 1, 379, 448, "relu2", True, False, True, "f32")])
def test_each_tile(counts, tokens, topk, n, k, act, gated, bias, slots, dt):
    run(counts, tokens, topk, n, k, act, gated, bias, slots, dt, seed=k)


@pytest.mark.parametrize("offset", [1, 2, 3])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_unaligned_outputs(offset, dt):
    for counts, tokens, n in (([4, 3], 4, 64), ([300, 200], 250, 64), ([90, 100], 100, 67)):
        run(counts, tokens, 2, n, 128, "relu2", True, True, False, dt, seed=9, offset=offset)


def test_extreme_sums():
    """All weights +1 and x = -128 over the longest row: the largest accumulator."""
    k, n = 131072, 33
    from oracle import bitnet_oracle as O
    packed = O.pack_codes(np.ones((n, k), np.int8))[None]
    w = N.TernaryExperts.from_packed(dev(packed), dev(np.array([0.5], F32)))
    for rows in (3, 200):
        r, _ = routing(np.zeros((rows, 1), np.int32), 1)
        x = np.full((rows, k), -128, np.int8)
        y = N.bitnet_expert_linear(r, w, dev(x), dev(np.ones(rows, F32)))
        assert (host(y) == -64.0 * k).all()


@pytest.mark.parametrize("act", ["relu2", "silu", "gelu"])
@pytest.mark.parametrize("n", [64, 24064])
def test_activations_over_their_range(act, n):
    """v = +-code * d, from 2^-40 to 2^60, dense around 0, through the kernels for few and many rows."""
    q = np.zeros((n, 64), np.int8)
    q[np.arange(n), np.arange(n) % 64] = 1 - 2 * (np.arange(n) // 64 % 2)
    from oracle import bitnet_oracle as O
    w = N.bitnet_repack_prefill(dev(O.pack_codes(q)))
    rows = 40 if n == 64 else 130
    x = np.random.default_rng(1).integers(-127, 128, (rows, 64)).astype(np.int8)
    d = np.r_[2.0 ** np.linspace(-40, 60, 10), np.linspace(1e-3, 0.3, rows - 10)].astype(F32)
    y = N.bitnet_ternary_linear_act(w, dev(np.ones(1, F32)), n, dev(x), dev(d), act=act)
    compare(y, *E.product(q, F32(1), x, d, act=act), "f32")


def test_a_thousand_experts():
    counts = np.zeros(1000, int)
    counts[[0, 3, 64, 500, 999]] = [1, 33, 2, 7, 40]
    run(list(counts), 83, 1, 33, 64, "relu2", True, False, False, "f32", seed=2)


def test_the_same_token_twice():
    """A pair list that names one expert twice gives the row twice."""
    e = np.array([[1, 1], [0, 1], [1, 1]], np.int32)
    y = run([1, 5], 3, 2, 40, 128, expert=e)
    assert torch.equal(y[1], y[2])


def test_contents_that_name_nothing():
    """Offsets past the batch or backwards, pairs past it or negative: other rows are right, nothing else is
    written."""
    xq, d = acts(6, 128, 1)
    q, g, w = matrices(3, 50, 128, 2)
    r, (first, pair, _) = routing(assign([4, 4, 4], 6, 2), 3)
    pair = pair.copy()
    pair[[1, 5]] = [-7, 1 << 30]
    r.pair.copy_(dev(pair))
    r.offset.copy_(torch.tensor([-5, 4, 8, 1 << 30], dtype=torch.int32))
    y = torch.full((12, 50), 7.0, device=DEV)
    N.bitnet_expert_linear(r, w, dev(xq), dev(d), y=y)
    for s in range(12):
        if s in (1, 5):
            assert (host(y[s]) == 7).all()
        else:
            row = pair[s] // 2
            same(y[s:s + 1], E.product(q[s // 4], g[s // 4], xq[row:row + 1], d[row:row + 1])[0], "f32")
    r.offset.copy_(torch.tensor([8, 4, 2, -1], dtype=torch.int32))      # empty experts only
    y.fill_(7.0)
    N.bitnet_expert_linear(r, w, dev(xq), dev(d), y=y)
    assert (host(y) == 7).all()


@pytest.mark.parametrize("m", [1, 2, 16, 17, 33, 64, 100, 200, 513])
@pytest.mark.parametrize("n,k", [(2560, 192), (129, 2560), (40, 64)])
def test_dense_is_the_prefill_product(m, n, k):
    xq, d = acts(m, k, m)
    _, g, w = matrices(1, n, k, 4)
    for dt in (torch.float32, torch.bfloat16):
        want = N.bitnet_ternary_linear_prefill([(w.w[0], w.scale, n)], dev(xq), dev(d), y_dtype=dt)[0]
        got = N.bitnet_ternary_linear_act(w.w[0], w.scale, n, dev(xq), dev(d), y_dtype=dt)
        assert torch.equal(got, want)


@pytest.mark.parametrize("gated,m,n", [(False, 3137, 4090), (True, 3130, 2043)])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_prompts(gated, m, n, dt):
    """Enough rows for the widest tile: against the plain products of the prefill call, whose epilogue in elementary
    operations rounds as the definition does."""
    k = 4160
    xq, d = acts(m, k, 1)
    x, dd = dev(xq), dev(d)
    g = torch.Generator(device=DEV).manual_seed(3)
    ws = [torch.randint(0, 256, (n, k // 4), generator=g, device=DEV, dtype=torch.uint8) for _ in range(1 + gated)]
    ws = [N.bitnet_repack_prefill(w & ~((w >> 1) & w & 0x55)) for w in ws]        # (no code 3)
    scale = torch.full((1,), 0.013, device=DEV)
    v = [N.bitnet_ternary_linear_prefill([(w, scale, n)], x, dd)[0] for w in ws]
    res = torch.randn(m, n, generator=g, device=DEV).to(dt)
    bias = torch.randn(n, generator=g, device=DEV)
    a = torch.relu(v[0] + bias)
    want = a * a
    if gated:
        want = want * v[1]
    got = N.bitnet_ternary_linear_act(ws[0], scale, n, x, dd, up=(ws[1], scale) if gated else None, bias=bias, act="relu2",
                                      residual=res, y_dtype=dt)
    assert torch.equal(got, (want + res.float()).to(dt))


@pytest.mark.parametrize("m", [1, 5, 40, 150, 300])
@pytest.mark.parametrize("act,gated", [("none", False), ("relu2", True), ("gelu", False), ("silu", True)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("wide", [0, 3200, 22400])
def test_dense_epilogue(m, act, gated, dt, wide):
    for n, bias, residual, offset in ((96, True, True, 0), (101, False, True, 0), (64, True, True, 1), (72, True, False, 0)):
        if wide and (m < 150 or n == 64 and wide > 4000):
            continue
        n += wide
        k = 320
        xq, d = acts(m, k, m)
        mats = [matrices(1, n, k, 6 + i) for i in range(1 + gated)]
        rng = np.random.default_rng(m + n)
        b = [rng.standard_normal(n).astype(F32) if bias else None for _ in mats]
        flat = torch.zeros(m * n + 8, dtype=TORCH[dt], device=DEV)
        res, rf = (None, None)
        if residual:
            t, rf = typed(2 * rng.standard_normal((m, n)), dt)
            res = flat[offset:offset + m * n].view(m, n)
            res.copy_(t)
        up = None if not gated else (mats[1][0][0], mats[1][1][0], b[1])
        want = E.product(mats[0][0][0], mats[0][1][0], xq, d, b[0], act, up, rf)
        args = dict(act=act, bias=None if not bias else dev(b[0]), up_bias=dev(b[1]) if gated and bias else None,
                    up=(mats[1][2].w[0], mats[1][2].scale) if gated else None, residual=res, y_dtype=TORCH[dt])
        w = mats[0][2]
        compare(N.bitnet_ternary_linear_act(w.w[0], w.scale, n, dev(xq), dev(d), **args), *want, dt)
        if residual:                                    # y in the residual's place
            y = N.bitnet_ternary_linear_act(w.w[0], w.scale, n, dev(xq), dev(d), **args, y=res)
            assert y is res
            compare(y, *want, dt)
            assert (flat[:offset] == 0).all() and (flat[offset + m * n:] == 0).all()


def test_nothing_to_do():
    _, _, w = matrices(2, 40, 128, 1)
    r = N.Routing.empty(0, 2, 2, DEV)
    assert N.bitnet_expert_linear(r, w, torch.empty((0, 128), dtype=torch.int8, device=DEV), torch.empty(0, device=DEV)).shape == (0, 40)
    r, _ = routing(np.full((40, 2), -1, np.int32), 2)          # a batch of padding
    xq, d = acts(40, 128, 1)
    y = torch.full((80, 40), 7.0, device=DEV)
    N.bitnet_expert_linear(r, w, dev(xq), dev(d), y=y)
    assert (host(y) == 7).all()


def test_another_stream():
    xq, d = acts(300, 192, 1)
    q, g, w = matrices(1, 70, 192, 2)
    x, dd = dev(xq), dev(d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = N.bitnet_ternary_linear_act(w.w[0], w.scale, 70, x, dd, act="relu2", stream=s)
    s.synchronize()
    same(y, E.product(q[0], g[0], xq, d, act="relu2")[0], "f32")
    packed = torch.randint(0, 3, (2, 40, 16), device=DEV, dtype=torch.uint8)
    torch.cuda.synchronize()
    again = N.TernaryExperts.from_packed(packed, torch.ones(2, device=DEV), stream=s)
    s.synchronize()
    for i in range(2):
        assert torch.equal(again.w[i], N.bitnet_repack_prefill(packed[i]))


def test_captured_products_follow_the_routing():
    """Two captured calls over one routing whose contents change between replays, with eager calls between."""
    experts, tokens, k, n = 5, 60, 192, 130
    q, g, w = matrices(experts, n, k, 3)
    xq, d = acts(tokens, k, 1)
    xs, ds = acts(tokens * 2, k, 2)
    x, dd, x2, d2 = dev(xq), dev(d), dev(xs), dev(ds)
    r = N.Routing.empty(tokens, 2, experts, DEV)
    r.expert.fill_(-1)
    N.bitnet_route(r)
    ys = [torch.zeros((tokens * 2, n), device=DEV) for _ in range(2)]
    calls = [lambda: N.bitnet_expert_linear(r, w, x, dd, act="relu2", y=ys[0]),
             lambda: N.bitnet_expert_linear(r, w, x2, d2, slots=True, y=ys[1])]
    graphs = []
    for f in calls:
        f()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f()
    for seed in range(4):
        e = assign([[0, 0, 120, 0, 0], [10, 20, 30, 40, 20], [1, 0, 0, 0, 2], [33, 0, 32, 31, 1]][seed], tokens, 2, seed)
        r.expert.copy_(dev(e))
        N.bitnet_route(r)
        for y in ys:
            y.fill_(7.0)
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        first, pair, _ = E.plan(e, experts)
        for i in range(experts):
            s0, s1 = first[i], first[i + 1]
            rows = pair[s0:s1] // 2
            if s1 > s0:
                same(ys[0][s0:s1], E.product(q[i], g[i], xq[rows], d[rows], act="relu2")[0], "f32")
                same(ys[1][s0:s1], E.product(q[i], g[i], xs[s0:s1], ds[s0:s1])[0], "f32")
        assert all((host(y[first[-1]:]) == 7).all() for y in ys)
        N.bitnet_expert_linear(r, w, x, dd)
        torch.cuda.synchronize()
