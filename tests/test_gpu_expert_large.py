"""Routing, experts' products and combination where offsets pass 32 bits (a few GB each)."""

import numpy as np
import pytest
import torch

from oracle import experts_oracle as E
from ternary_weight_linear_bit_amd import _native as N

from experts_util import acts, dev, host, matrices, same
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.lib()


@pytest.fixture(autouse=True)
def _memory():
    yield
    torch.cuda.empty_cache()


def test_gathered_rows_up_to_2_31_bytes():
    tokens, k, n = 1 << 20, 2048, 40
    at = [0, 1 << 19, tokens - 2, tokens - 1]
    x, d = torch.zeros((tokens, k), dtype=torch.int8, device=DEV), torch.ones(tokens, device=DEV)
    xq, ds = acts(len(at), k, 1)
    x[at], d[at] = dev(xq), dev(ds)
    q, g, w = matrices(2, n, k, 1)
    r = N.Routing.empty(tokens, 1, 2, DEV)
    r.expert.fill_(-1)
    r.expert[at] = torch.tensor([[0], [1], [1], [0]], dtype=torch.int32, device=DEV)
    N.bitnet_route(r)
    y = torch.full((tokens, n), 7.0, device=DEV)
    N.bitnet_expert_linear(r, w, x, d, y=y)
    assert host(r.offset).tolist() == [0, 2, 4]
    for slot, (e, i) in enumerate(((0, 0), (0, 3), (1, 1), (1, 2))):
        same(y[slot:slot + 1], E.product(q[e], g[e], xq[i:i + 1], ds[i:i + 1])[0], "f32")
    assert bool((y[4:] == 7).all())


def test_rows_by_slot_past_2_32_bytes():
    pairs, k, n = (1 << 19) + 3, 8256, 33
    at = [0, 260000, pairs - 2, pairs - 1]
    x, d = torch.zeros((pairs, k), dtype=torch.int8, device=DEV), torch.ones(pairs, device=DEV)
    xq, ds = acts(len(at), k, 2)
    x[at], d[at] = dev(xq), dev(ds)
    q, g, w = matrices(1, n, k, 2)
    r = N.Routing.empty(pairs, 1, 1, DEV)
    r.offset.copy_(torch.tensor([0, pairs], dtype=torch.int32))
    y = N.bitnet_expert_linear(r, w, x, d, slots=True)
    same(y[at], E.product(q[0], g[0], xq, ds)[0], "f32")


@pytest.mark.parametrize("k", [64, 192])
def test_outputs_past_2_32_values(k):
    m, n = (1 << 20) + 5, 4104
    x = torch.randint(-128, 128, (m, k), device=DEV, dtype=torch.int8)
    d = torch.rand(m, device=DEV)
    q, g, w = matrices(1, n, k, 3)
    y = N.bitnet_ternary_linear_act(w.w[0], w.scale, n, x, d, act="relu2", y_dtype=torch.bfloat16)
    for at in (slice(0, 3), slice(1 << 19, (1 << 19) + 2), slice(m - 70, m)):
        same(y[at], E.product(q[0], g[0], host(x[at]), host(d[at]), act="relu2")[0], "bf16")


def test_combined_rows_past_2_32_values():
    m, k = (1 << 20) + 3, 4104
    r = N.Routing.empty(m, 1, 1, DEV)
    r.slot.copy_(torch.arange(m - 1, -1, -1, device=DEV, dtype=torch.int32)[:, None])
    r.weight.fill_(0.5)
    y = torch.zeros((m, k), dtype=torch.bfloat16, device=DEV)
    y[0], y[m - 1], y[m - 2] = 3.0, 5.0, 7.0
    out = N.bitnet_combine(r, y)
    assert bool((out[m - 1] == 1.5).all()) and bool((out[0] == 2.5).all()) and bool((out[1] == 3.5).all())
    assert int(torch.count_nonzero(out[2:m - 1])) == 0


def test_logits_past_2_32_values():
    tokens, experts, topk = (1 << 22) + 9, 1024, 2
    x = torch.randn((1 << 12, experts), device=DEV).to(torch.bfloat16)
    x = x.repeat((tokens + x.shape[0] - 1) // x.shape[0], 1)[:tokens]
    r = N.bitnet_route(N.Routing.empty(tokens, topk, experts, DEV), x, "chosen")
    for at in (slice(0, 5), slice(1 << 21, (1 << 21) + 5), slice(tokens - 5, tokens)):
        np.testing.assert_array_equal(host(r.expert[at]), E.choose(x[at].float().cpu().numpy(), topk))
    flat = r.expert.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    assert torch.equal(r.pair.long(), order)
    assert torch.equal(r.slot.reshape(-1)[order].long(), torch.arange(flat.numel(), device=DEV))
    count = torch.bincount(flat, minlength=experts)
    assert torch.equal(r.offset[1:].long(), count.cumsum(0)) and int(r.offset[0]) == 0
