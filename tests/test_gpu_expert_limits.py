"""Products, offsets and combination at the largest sizes that the calls take (up to 90 GB)."""

import numpy as np
import pytest
import torch

from oracle import bitnet_oracle as O
from oracle import experts_oracle as E
from ternary_weight_linear_bit_amd import _native as N
from ternary_weight_linear_bit_amd import inputs as I

from experts_util import F32, acts, dev, matrices, same
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


def block(seed):
    """32 x 64 weights and their block of the prefill layout."""
    q = I.ternary_codes(32, 64, seed)
    return q, N.bitnet_repack_prefill(dev(O.pack_codes(q)))[0]


@pytest.mark.parametrize("gated,n", [(False, 2 ** 31 - 32), (True, 2 ** 31 - 1152)])
def test_most_outputs_of_a_row(gated, n):
    """The largest N, which with a tile's width passes 31 bits, and the largest that gate and up leave a launch: one
    block of weights everywhere but for some at the beginning, the end and in between."""
    rows = 2
    q, one = block(1)
    w = torch.empty(N.prefill_layout_shape(n, 64), dtype=torch.uint8, device=DEV)
    w.copy_(one.expand_as(w))
    others = {0: 2, 2 ** 25: 3, n // 32 - 9: 4, n // 32 - 2: 5, n // 32 - 1: 6}
    for at, seed in others.items():
        w[at] = block(seed)[1]
    xq, d = acts(rows, 64, 1)
    scale = torch.full((1,), 0.5, device=DEV)
    buf = torch.full((rows * n + 32,), 7.0, dtype=torch.bfloat16, device=DEV)
    y = buf[:rows * n].view(rows, n)
    print("weights laid out", flush=True)
    N.bitnet_ternary_linear_act(w, scale, n, dev(xq), dev(d), up=(w, scale) if gated else None, act="relu2", y=y)
    torch.cuda.synchronize()

    def want(q):
        up = (q, F32(0.5), None) if gated else None
        a = E.bf16(E.product(q, F32(0.5), xq, d, act="relu2", up=up)[0])
        return torch.from_numpy(a).to(torch.bfloat16).to(DEV)
    blocks = y.view(rows, n // 32, 32)
    for at, seed in others.items():
        assert torch.equal(blocks[:, at], want(block(seed)[0])), at
        blocks[:, at] = want(q)
    for m in range(rows):
        assert bool((blocks[m] == want(q)[m]).all())
    assert bool((buf[rows * n:] == 7).all())


def test_overlapping_ranges_of_many_slots():
    """Every second expert's range is the whole batch: 512 times its tiles, more than 2^31, are no tiles of a plan.  The
    matrices are alike, so that a slot's values are the same whichever expert it goes to."""
    pairs, experts, n = 2 ** 29 - 40000, 1024, 8
    x, d = torch.zeros((pairs, 64), dtype=torch.int8, device=DEV), torch.ones(pairs, device=DEV)
    at = [0, 12345, 1 << 28, pairs - 97, pairs - 1]
    xq, ds = acts(len(at), 64, 1)
    x[at], d[at] = dev(xq), dev(ds)
    q, g, w = matrices(1, n, 64, 3)
    w = N.TernaryExperts(w.w.repeat(experts, 1, 1), w.scale.repeat(experts), n, 64)
    none = torch.empty((pairs, 1), dtype=torch.int32, device=DEV)      # (not read by slot)
    offset = torch.tensor([0, pairs], dtype=torch.int32, device=DEV).repeat(experts // 2 + 1)[:experts + 1]
    r = N.Routing(none, none.view(torch.float32), offset, none.view(-1), none)
    y = torch.full((pairs, n), 7.0, dtype=torch.bfloat16, device=DEV)
    print("batch laid out", flush=True)
    N.bitnet_expert_linear(r, w, x, d, slots=True, y=y)
    torch.cuda.synchronize()
    same(y[at], E.product(q[0], g[0], xq, ds)[0], "bf16")
    y[at] = 0.0
    assert int(torch.count_nonzero(y)) == 0


@pytest.mark.parametrize("k,tokens", [(3, 2 ** 24 + 300), (8, 2 ** 24 + 300), (2 ** 23 - 1, 520)])
@pytest.mark.parametrize("residual", [False, True])
def test_combined_tokens_beyond_the_grid(k, tokens, residual):
    """More tokens than the grid's first dimension has workgroups: 2^24 - 1 of them for rows of one part, narrow or in
    16 bytes, and 511 beside the 32768 parts of the longest rows."""
    r = N.Routing.empty(tokens, 1, 1, DEV)
    r.slot.copy_(torch.arange(tokens - 1, -1, -1, device=DEV, dtype=torch.int32)[:, None])
    r.slot[[1, tokens - 2]] = -1
    r.weight.fill_(2.0)
    v = (torch.arange(tokens, device=DEV) % 85).to(torch.bfloat16)          # a row's values; up to 3 * 84 they are exact in bf16
    y = v[:, None].expand(tokens, k).contiguous()
    want = 2 * v.flip(0)
    want[[1, tokens - 2]] = 0
    base = None
    if residual:
        base = y.clone() if k < 100 else y
        want += v
    out = N.bitnet_combine(r, y, base, out=torch.full_like(y, 7.0))
    for m in range(0, tokens, 1 << 22):
        assert bool((out[m:m + (1 << 22)] == want[m:m + (1 << 22), None]).all()), m
