"""bitnet_attention on rows whose weights differ by many orders: a key far above thousands of
others, and outputs that are single weights.  Both kernels, all types, bounds that look at each
weight by itself (attention_rows.weight_bounds)."""

import numpy as np
import pytest
import torch

from oracle import layer_oracle as L
from ternary_weight_linear_bit_amd import _native as N

from attention_rows import one_key_a_dim, paged, peaked, weight_bounds
from gpu_helpers import DEV, dev, host

pytestmark = pytest.mark.gpu
F32 = np.float32
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
PAIRS = pytest.mark.parametrize("dt,out_dt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
# kv heads, query heads, rows of a sequence, the least stated max_len: 16 columns a workgroup
# and few heads for the decode kernel; 48 columns and a large cache for the prompt kernel
DECODE, PROMPT = (2, 6, 2, 0), (32, 32, 50, 16384)
BOTH = pytest.mark.parametrize("size", [DECODE, PROMPT], ids=["decode", "prompt"])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.lib()


def run(size, dim, page, lens, dt, out_dt, gap, at=0, value=(False, True), spread=1.0, alone="", window=0,
        seed=0, rows=None, holes=0.0):
    heads, q_heads, new, least = size
    new = rows or new
    rng = np.random.default_rng(500 + seed)
    made = [peaked(rng, new, q_heads, heads, dim, n, gap, at, value, spread) for n in lens]
    qf = np.concatenate([m[0] for m in made])
    ks, vs, table, first = [], [], np.full((len(lens), max(-(-max(lens) // page), least // page)), -1, np.int32), 0
    for b, m in enumerate(made):
        large = [[(at + i) % lens[b] for i in range(q_heads) if i // (q_heads // heads) == h] for h in range(heads)]
        vc = one_key_a_dim(rng, lens[b], dim, heads, None if alone == "all" else large) if alone else m[2]
        k, v = paged(m[1], vc, page)
        table[b, :len(k)] = first + rng.permutation(len(k))
        ks.append(np.empty_like(k))
        vs.append(np.empty_like(v))
        ks[-1][table[b, :len(k)] - first], vs[-1][table[b, :len(k)] - first] = k, v
        first += len(k)
    if holes:                                             # pages that are not there
        table[rng.random(table.shape) < holes] = 1 << 20
    k, v = np.concatenate(ks), np.concatenate(vs)
    dk, dv, scale = made[0][3:]
    dks, dvs = np.full((first, heads), dk, F32), np.full((first, heads), dv, F32)
    q_start = np.arange(len(lens) + 1, dtype=np.int32) * new
    kv_len = np.asarray(lens, np.int32)
    max_len = table.shape[1] * page
    c = N.KVCache(dev(k), dev(v), dev(dks), dev(dvs))
    b = N.KVBatch(dev(table), dev(q_start), dev(kv_len), new, max_len)
    q = dev(qf).to(TYPES[dt])
    out = torch.empty(q.shape, dtype=TYPES[out_dt], device=DEV)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=DEV)
    N.bitnet_attention(c, b, q, scale=float(scale), window=window, out=out, lse=lse)
    got, gl = host(out.float()), host(lse)
    want, wl, *detail = L.attention(k, v, dks, dvs, table, q_start, kv_len, qf, scale, window, new, max_len,
                                    detail=True)
    none = np.isneginf(wl)                                # rows whose keys are all missing
    assert np.all(got[none] == 0) and np.array_equal(np.isneginf(gl), none)
    wl, gl = np.where(none, 0, wl), np.where(none, 0, gl)
    keys = np.repeat(kv_len, new)[:, None].astype(np.float64)
    tol, tol_l = weight_bounds(want, wl, *detail, qf, keys, dt == "f32" and out_dt == "f32", out_dt == "bf16",
                               steps=0 if size is DECODE else keys / 64 + 1)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (bad.mean(), np.max(np.abs(got - want) / tol), np.argwhere(bad)[:5], got[bad][:5],
                           want[bad][:5], tol[bad][:5])
    assert np.all(np.abs(gl - wl) <= tol_l), np.max(np.abs(gl - wl) / tol_l)


@BOTH
@PAIRS
@pytest.mark.parametrize("gap", [0, 6, 9, 12, 14, 18, 30])
def test_one_key_above_many(size, dt, out_dt, gap):
    """The first keys outweigh the others, every second of them without a value."""
    run(size, 128, 64, [64, 1024, 8191] if size is DECODE else [300, 4000], dt, out_dt, gap, seed=gap)


@BOTH
@PAIRS
@pytest.mark.parametrize("at", [700, 2040, -6])
def test_where_the_key_lies(size, dt, out_dt, at):
    """In the middle, before a step's end, among the last keys (which some rows do not see)."""
    run(size, 64, 16, [2047, 2049], dt, out_dt, 13, at=at, seed=at % 7)


@BOTH
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [16, 80, 256])
def test_other_widths(size, dt, dim):
    run(size, dim, 32, [129, 900], dt, dt, 12, value=(False,), seed=dim)


@BOTH
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_window_past_the_key(size, dt):
    """Rows that see the key, and rows whose window has left it behind."""
    run(size, 64, 16, [400, 430], dt, dt, 14, at=350 if size is PROMPT else 398, window=40, seed=3)


@BOTH
@PAIRS
@pytest.mark.parametrize("spread", [0.3, 1.5, 5.0, 9.0])
def test_each_weight_by_itself(size, dt, out_dt, spread):
    """Every dim has the value of one key only: its output is that key's weight, down to 2^-48 of
    the largest."""
    run(size, 128, 64, [100, 300], dt, out_dt, 5, at=40, spread=spread, alone="all", seed=int(spread))


@BOTH
@PAIRS
@pytest.mark.parametrize("gap,spread", [(3, 0.5), (9, 0.5), (14, 1.5), (14, 4.0), (22, 0.5), (22, 1.5), (30, 0.5)])
def test_each_small_weight_by_itself(size, dt, out_dt, gap, spread):
    """The same, where no dim has a value of the keys that outweigh the others."""
    run(size, 128, 64, [100, 300], dt, out_dt, gap, at=3, spread=spread, alone="small", seed=gap)
    run(size, 64, 16, [70, 90], dt, out_dt, gap, at=30, spread=spread, alone="small", seed=gap, window=60)


@pytest.mark.parametrize("dt,out_dt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("gap", [10, 14])
def test_long_caches(dt, out_dt, gap):
    """65536 keys in many parts, the key in one of them."""
    run((1, 4, 1, 0), 128, 128, [65536], dt, out_dt, gap, value=(False, True), seed=gap)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_one_workgroup_of_eight_waves(dt):
    """Up to 512 keys: a step for each wave."""
    run(DECODE, 128, 64, [512, 300, 65], dt, dt, 14, seed=5)


@pytest.mark.parametrize("out_dt", ["bf16", "f32"])
@pytest.mark.parametrize("gap,alone", [(14, ""), (22, "small")])
def test_wide_prompts(out_dt, gap, alone):
    """Enough bf16 columns for workgroups of 256."""
    run((256, 256, 130, 0), 128, 64, [200], "bf16", out_dt, gap, at=3, alone=alone, seed=gap)


@pytest.mark.parametrize("size,dim,page,lens,dt,out_dt,at,value,spread,alone,seed", [
    ((2, 2, 1, 4096), 192, 16, [2362, 84], "f32", "f32", -3, (False,), 2, "small", 324073),
    ((2, 8, 1, 0), 256, 16, [323, 91], "bf16", "f32", 0, (True,), 8, "all", 308241),
    ((1, 7, 1, 0), 96, 64, [1286, 558, 141], "f32", "bf16", 0, (False, True), 4, "all", 483414),
    ((1, 1, 5, 0), 160, 32, [1377, 657], "bf16", "f32", 0, (True,), 2, "all", 898264)])
def test_smallest_weights_that_count(monkeypatch, size, dim, page, lens, dt, out_dt, at, value, spread, alone, seed):
    """Outputs that are weights just above 2^-48 of the row's largest."""
    monkeypatch.setattr(f"{__name__}.DECODE", size)
    run(size, dim, page, lens, dt, out_dt, 30, at=at, value=value, spread=spread, alone=alone, seed=seed)


@BOTH
@pytest.mark.parametrize("dt,out_dt", [("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("gap,alone", [(12, ""), (22, "small")])
def test_missing_pages(size, dt, out_dt, gap, alone):
    """Pages that are not there among those with the keys that count, and rows left with none."""
    run(size, 64, 16, [90, 700], dt, out_dt, gap, at=20, alone=alone, holes=0.3, seed=gap)
    run(size, 128, 64, [64, 300], dt, out_dt, gap, at=70, alone=alone, holes=0.5, seed=gap + 4, window=90)


@pytest.mark.parametrize("size", [DECODE, PROMPT], ids=["decode", "prompt"])
def test_captured_beside_eager_calls(size):
    """A graph replayed over rows with and without a dominant key, eager calls in between."""
    heads, q_heads, new, least = size
    rng = np.random.default_rng(1)
    made = [peaked(rng, new, q_heads, heads, 64, 400, gap, 9, (False, True)) for gap in (0, 13, 22)]
    pages = [paged(m[1], m[2], 16) for m in made]
    n, width = 25, max(25, least // 16)
    table = np.full((1, width), -1, np.int32)
    table[0, :n] = rng.permutation(n)
    scales = np.full((n, heads), made[0][3], F32), np.full((n, heads), made[0][4], F32)
    c = N.KVCache(torch.empty((n, heads, 16, 64), dtype=torch.int8, device=DEV),
                  torch.empty((n, heads, 64, 16), dtype=torch.int8, device=DEV), dev(scales[0]), dev(scales[1]))
    b = N.KVBatch(dev(table), dev(np.array([0, new], np.int32)), dev(np.array([400], np.int32)), new, width * 16)
    q = torch.zeros((new, q_heads, 64), dtype=torch.bfloat16, device=DEV)
    scale = float(made[0][5])

    def fill(i):
        at = torch.from_numpy(table[0, :n].astype(np.int64)).to(DEV)
        c.k[at], c.v[at] = dev(pages[i][0]), dev(pages[i][1])
        q.copy_(dev(made[i][0]))
    fill(0)
    N.bitnet_attention(c, b, q, scale=scale)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = N.bitnet_attention(c, b, q, scale=scale)
    for i in (1, 0, 2, 1, 2):
        fill(i)
        g.replay()
        assert torch.equal(out, N.bitnet_attention(c, b, q, scale=scale)) and bool(out.any())


@BOTH
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_least_value_scales(monkeypatch, size, dt):
    """Values of scale 2^-40 beside a dominant key: neither sum leaves fp32's range."""
    real = peaked

    def tiny(*a, **kw):
        q, kc, vc, dk, _, scale = real(*a, **kw)
        return q, kc, vc, dk, F32(2.0 ** -40), scale
    monkeypatch.setattr(f"{__name__}.peaked", tiny)
    for gap in (0, 22, 40):
        run(size, 64, 16, [300, 1500], dt, "f32", gap, seed=gap)
