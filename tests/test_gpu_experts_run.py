"""A decoder layer's feed-forward of experts through the library's calls, as a program runs it:
act-quant, routing, gate and up, act-quant, down, combination, residual join; eager, captured and replayed."""

import numpy as np
import pytest
import torch

from oracle import bitnet_oracle as O
from oracle import experts_oracle as E
from ternary_weight_linear_bit_amd import _native as N
from ternary_weight_linear_bit_amd import inputs as I

from experts_util import F32, dev, host, matrices, same
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu
HIDDEN, WIDTH, EXPERTS, TOPK = 256, 192, 7, 2


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.lib()


class Layer:
    def __init__(self):
        self.gate, self.up = matrices(EXPERTS, WIDTH, HIDDEN, 1), matrices(EXPERTS, WIDTH, HIDDEN, 2)
        self.down = matrices(EXPERTS, HIDDEN, WIDTH, 3)
        self.shared = [matrices(1, n, k, 7 + i) for i, (n, k) in enumerate(((WIDTH, HIDDEN), (WIDTH, HIDDEN), (HIDDEN, WIDTH)))]
        self.norm = I.norm_weight(HIDDEN, 5)
        self.norm_dev = dev(self.norm)

    def gpu(self, x, logits, h, r):
        """x [M, HIDDEN] bf16, router logits, residual stream h fp32: the new stream and its codes."""
        xq, d = N.bitnet_quantize_acts(x)
        N.bitnet_route(r, logits, "chosen")
        a = N.bitnet_expert_linear(r, self.gate[2], xq, d, up=self.up[2], act="relu2", y=self.inner(r))
        aq, ad = N.bitnet_quantize_acts(a)
        y = N.bitnet_expert_linear(r, self.down[2], aq, ad, slots=True, y_dtype=torch.bfloat16)
        # an expert that every token passes through, its output under the others' sum
        g, u, o = (m[2] for m in self.shared)
        s = N.bitnet_ternary_linear_act(g.w[0], g.scale, WIDTH, xq, d, up=(u.w[0], u.scale), act="relu2", y_dtype=torch.bfloat16)
        sq, sd = N.bitnet_quantize_acts(s)
        base = N.bitnet_ternary_linear_act(o.w[0], o.scale, HIDDEN, sq, sd, y_dtype=torch.bfloat16)
        z = N.bitnet_combine(r, y, base, out=base)
        return N.bitnet_residual_norm(z, h, pre_weight=self.norm_dev)

    def inner(self, r):
        return torch.zeros((r.tokens * r.topk, WIDTH), dtype=torch.bfloat16, device=DEV)

    def oracle(self, x, logits):
        xq, d = O.quantize_acts(x)
        expert = E.choose(logits, TOPK)
        offset, pair, slot = E.plan(expert, EXPERTS)
        y = np.zeros((expert.size, HIDDEN), F32)

        def feed(gate, up, down, e, xq, d):
            inner = E.bf16(E.product(gate[0][e], gate[1][e], xq, d, None, "relu2", (up[0][e], up[1][e], None))[0])
            q, s = O.quantize_acts(inner)
            return E.bf16(E.product(down[0][e], down[1][e], q, s)[0])
        for e in range(EXPERTS):
            s0, s1 = offset[e], offset[e + 1]
            if s1 > s0:
                rows = pair[s0:s1] // TOPK
                y[s0:s1] = feed(self.gate, self.up, self.down, e, xq[rows], d[rows])
        base = feed(*self.shared, 0, xq, d)
        return expert, y, base, slot


def inputs(m, seed):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.standard_normal((m, HIDDEN)).astype(F32)).to(torch.bfloat16)
    logits = rng.standard_normal((m, EXPERTS)).astype(F32)
    logits[m - m // 5:] = -np.inf               # padding
    h = rng.standard_normal((m, HIDDEN)).astype(F32)
    return x, logits, h


def verify(layer, x, logits, h, got, r):
    expert, y, base, slot = layer.oracle(x.float().numpy(), logits)
    np.testing.assert_array_equal(host(r.expert), expert)
    np.testing.assert_array_equal(host(r.slot), slot)
    z = E.bf16(E.combine(host(r.weight), slot, y, base))
    out = (h + z).astype(F32)
    same(got[0], out, "f32")
    u = O.rms_normalise(out, layer.norm, 1e-5)
    q, s = O.quantize_acts(u)
    np.testing.assert_array_equal(host(got[1]), q)
    np.testing.assert_array_equal(host(got[2]).view(np.uint32), s.view(np.uint32))


@pytest.mark.parametrize("m", [1, 7, 60, 700])
def test_layer(m):
    layer = Layer()
    x, logits, h = inputs(m, m)
    r = N.Routing.empty(m, TOPK, EXPERTS, DEV)
    got = layer.gpu(x.to(DEV), dev(logits), dev(h), r)
    verify(layer, x, logits, h, got, r)


@pytest.mark.parametrize("m", [5, 300])
def test_captured_layer(m):
    layer = Layer()
    x, logits, h = inputs(m, 1)
    xt, lt, ht = x.to(DEV), dev(logits), dev(h)
    r = N.Routing.empty(m, TOPK, EXPERTS, DEV)
    layer.gpu(xt, lt, ht, r)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = layer.gpu(xt, lt, ht, r)
    for seed in (2, 3, 4):
        x, logits, h = inputs(m, seed)
        xt.copy_(x.to(DEV))
        lt.copy_(dev(logits))
        ht.copy_(dev(h))
        g.replay()
        torch.cuda.synchronize()
        verify(layer, x, logits, h, got, r)
        other = N.Routing.empty(m, TOPK, EXPERTS, DEV)
        layer.gpu(xt, lt, ht, other)
        torch.cuda.synchronize()
