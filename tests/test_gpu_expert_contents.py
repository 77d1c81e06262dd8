"""Experts' products over routings whose contents no plan has, or change between replays, at sizes that the kernel for
few rows takes and each tile of the one for many."""

import numpy as np
import pytest
import torch

from oracle import experts_oracle as E
from ternary_weight_linear_bit_amd import _native as N

from experts_util import acts, assign, dev, host, matrices, routing, same
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

EXPERTS, K = 3, 192
# slots, N, gate and up: few rows; tiles of 32 slots with the k steps shared by eight and by four groups; of 32, 64, 96 slots
SIZES = [(150, 300, False), (150, 300, True), (150, 1355, False), (150, 1355, True), (150, 5364, False), (150, 15914, True),
         (600, 8107, True)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.lib()


class Case:
    def __init__(self, slots, n, gated):
        self.slots, self.tokens, self.n, self.gated = slots, slots // 2, n, gated
        self.x, self.d = acts(self.tokens, K, 1)
        self.xs, self.ds = acts(slots, K, 2)
        self.mats = [matrices(EXPERTS, n, K, 3 + i) for i in range(1 + gated)]
        self.on = [tuple(map(dev, a)) for a in ((self.x, self.d), (self.xs, self.ds))]

    def call(self, r, by_slot, y):
        N.bitnet_expert_linear(r, self.mats[0][2], *self.on[by_slot], slots=bool(by_slot), act="relu2",
                               up=self.mats[1][2] if self.gated else None, y=y)

    def want(self, e, rows, by_slot):
        x, d = ((self.x, self.d), (self.xs, self.ds))[by_slot]
        up = (self.mats[1][0][e], self.mats[1][1][e], None) if self.gated else None
        return E.product(self.mats[0][0][e], self.mats[0][1][e], x[rows], d[rows], act="relu2", up=up)[0]

    def empty(self):
        return torch.full((self.slots, self.n), 7.0, device=DEV)


@pytest.mark.parametrize("slots,n,gated", SIZES)
def test_contents_that_name_nothing(slots, n, gated):
    """Offsets before and past the batch, pairs of no token: other rows are right, nothing else is written.  Offsets
    that go backwards are empty experts."""
    c = Case(slots, n, gated)
    third = slots // 3
    r, (_, pair, _) = routing(assign([third] * 3, c.tokens, 2), EXPERTS)
    bad = {1: -7, 5: 1 << 30, third: -1 << 31, 2 * third + 1: (1 << 31) - 1, slots - 1: slots}
    pair = pair.copy()
    pair[list(bad)] = list(bad.values())
    r.pair.copy_(dev(pair))
    r.offset.copy_(torch.tensor([-5, third, 2 * third, 1 << 30], dtype=torch.int32))
    for by_slot in (0, 1):
        y = c.empty()
        c.call(r, by_slot, y)
        for e in range(EXPERTS):
            s = np.arange(e * third, (e + 1) * third)
            s = s if by_slot else s[~np.isin(s, list(bad))]
            same(y[torch.from_numpy(s).to(DEV)], c.want(e, s if by_slot else pair[s] // 2, by_slot), "f32")
        if not by_slot:
            assert (host(y)[list(bad)] == 7).all()
    for offset in ([2 * third, third, 7, -1], [slots, 1 << 30, slots + 1, -5], [0, 0, 0, 0], [-1, -2, -(1 << 31), 0]):
        r.offset.copy_(torch.tensor(offset, dtype=torch.int32))
        y = c.empty()
        for by_slot in (0, 1):
            c.call(r, by_slot, y)
        assert bool((y == 7).all()), offset


@pytest.mark.parametrize("slots,n,gated", SIZES)
def test_overlapping_ranges(slots, n, gated):
    """A slot in two experts' ranges gets values of one or the other, the rest their own expert's."""
    c = Case(slots, n, gated)
    r, (_, pair, _) = routing(np.zeros((c.tokens, 2), np.int32), EXPERTS)
    a, b = slots // 2 + 10, slots // 2 - 10
    r.offset.copy_(torch.tensor([0, a, b, slots], dtype=torch.int32))
    for by_slot in (0, 1):
        y = c.empty()
        c.call(r, by_slot, y)
        rows = np.arange(slots) if by_slot else pair // 2
        same(y[:b], c.want(0, rows[:b], by_slot), "f32")
        same(y[a:], c.want(2, rows[a:], by_slot), "f32")
        both = host(y[b:a])
        assert ((both == c.want(0, rows[b:a], by_slot)) | (both == c.want(2, rows[b:a], by_slot))).all()


@pytest.mark.parametrize("slots,n,gated", SIZES)
def test_captured_products_follow_the_routing(slots, n, gated):
    """Two captured calls over one routing, from one busy expert to all of them to next to none, with eager calls over
    another between the replays."""
    c = Case(slots, n, gated)
    r = N.Routing.empty(c.tokens, 2, EXPERTS, DEV)
    r.expert.fill_(-1)
    N.bitnet_route(r)
    ys = [c.empty(), c.empty()]
    graphs = []
    for by_slot in (0, 1):
        c.call(r, by_slot, ys[by_slot])
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c.call(r, by_slot, ys[by_slot])
    assert all(bool((y == 7).all()) for y in ys)            # a batch of padding
    other, _ = routing(assign([slots // 3] * 3, c.tokens, 2), EXPERTS)
    for seed, counts in enumerate(([0, slots, 0], [slots // 3] * 3, [1, 0, 2], [33, slots - 65, 32], [0, 0, 0], [64, 1, 0])):
        e = assign(counts, c.tokens, 2, seed)
        r.expert.copy_(dev(e))
        N.bitnet_route(r)
        for y in ys:
            y.fill_(7.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        first, pair, _ = E.plan(e, EXPERTS)
        for i in range(EXPERTS):
            s = np.arange(first[i], first[i + 1])
            if s.size:
                same(ys[0][s[0]:s[-1] + 1], c.want(i, pair[s] // 2, 0), "f32")
                same(ys[1][s[0]:s[-1] + 1], c.want(i, s, 1), "f32")
        assert all(bool((y[int(first[-1]):] == 7).all()) for y in ys)
        c.call(other, seed % 2, c.empty())
        torch.cuda.synchronize()
