"""bitnet_attention on the GPU against float64, within bounds derived from the types
(layer_util.attention_bounds)."""

import numpy as np
import pytest
import torch

from oracle import layer_oracle as L
from ternary_weight_linear_bit_amd import _native as N

from gpu_helpers import DEV, dev, host
from layer_util import attention_bounds, cache, seqs

pytestmark = pytest.mark.gpu
F32 = np.float32
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.lib()


def run(heads, q_heads, dim, page, news, lens, dt="bf16", out_dt=None, window=0, seed=0, tail=0,
        edit=None, scale=None, sharp=1.0, max_new=None, strided=False, flood=True, max_len=None):
    out_dt = out_dt or dt
    rng = np.random.default_rng(200 + seed)
    q_start, kv_len, table, pages = seqs(news, lens, page, seed=seed)
    T = int(q_start[-1]) + tail
    k, v, ks, vs = cache(pages, heads, page, dim, seed)
    if edit:
        edit(table, q_start, kv_len, ks, vs)
    used = np.unique(table[table >= 0])
    if flood:   # pages of no sequence, as fresh memory may hold them
        idle = np.setdiff1d(np.arange(pages), used)
        ks[idle], vs[idle] = np.nan, np.inf
    q = rng.standard_normal((T, q_heads, dim)) * sharp
    qt = torch.from_numpy(q.astype(F32)).to(TYPES[dt])
    qf = qt.float().numpy()
    if T > int(q_start[-1]) and not edit:
        qt[int(q_start[-1]):] = float("nan")          # rows of nobody
    if strided:
        wide = torch.full((T, q_heads * dim + 24), 9.0, dtype=TYPES[dt])
        wide[:, 8:8 + q_heads * dim] = qt.reshape(T, -1)
        qt = wide.to(DEV)[:, 8:8 + q_heads * dim].unflatten(1, (q_heads, dim))
    else:
        qt = qt.to(DEV)
    most = max(news) if max_new is None else max_new
    max_len = table.shape[1] * page if max_len is None else max_len
    c = N.KVCache(dev(k), dev(v), dev(ks), dev(vs))
    b = N.KVBatch(dev(table), dev(q_start), dev(kv_len), most, max_len)
    out = torch.full((T, q_heads, dim), 7.0, dtype=TYPES[out_dt], device=DEV)
    lse = torch.full((T, q_heads), 7.0, dtype=torch.float32, device=DEV)
    scale = dim ** -0.5 if scale is None else scale
    assert N.bitnet_attention(c, b, qt, scale=scale, window=window, out=out, lse=lse) is out
    want, wl, absv, flat, top, reach = L.attention(k, v, ks, vs, table, q_start, kv_len, qf, F32(scale),
                                                   window, most, max_len, detail=True)
    got, gl = host(out.float()), host(lse)
    none = np.isnan(want)
    assert np.all(got[none] == 7.0) and np.all(gl[np.isnan(wl)] == 7.0)     # left as they were
    empty = np.isneginf(wl)
    assert np.all(got[empty] == 0.0) and np.all(np.isneginf(gl[empty]))
    exact_io = dt == "f32" and out_dt == "f32"
    keys = np.full(wl.shape, float(max(lens)))
    tol, tol_l = attention_bounds(np.nan_to_num(want), np.where(np.isnan(wl), 0, wl), absv, flat, top, reach,
                                  np.nan_to_num(qf), keys, exact_io)
    assert np.all(np.isfinite(got))
    bad = ~none & ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], tol[bad][:5])
    badl = np.isfinite(wl) & ~(np.abs(gl - np.where(np.isfinite(wl), wl, 0)) <= tol_l)
    assert not badl.any(), (np.argwhere(badl)[:5], gl[badl][:5], wl[badl][:5], tol_l[badl][:5])
    return got


SHAPES = [(5, 20, 128), (2, 2, 64), (1, 1, 16), (2, 6, 80), (1, 2, 256), (1, 24, 128), (1, 5, 48), (2, 80, 32)]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("heads,q_heads,dim", SHAPES)
def test_single_tokens(heads, q_heads, dim, page, dt):
    """One new token each, at lengths around every boundary, none and one among them."""
    lens = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 700]
    run(heads, q_heads, dim, page, [1] * len(lens), lens, dt, seed=page + dim)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("heads,q_heads,dim", SHAPES)
def test_few_rows(heads, q_heads, dim, page, dt):
    """Drafted tokens: several rows a sequence, idle sequences between."""
    run(heads, q_heads, dim, page, [3, 0, 1, 7, 2, 5], [3, 9, 40, 200, 2, 130], dt, seed=page + dim)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("heads,q_heads,dim", [(1, 4, 128), (2, 2, 64), (1, 3, 80), (1, 1, 256), (1, 20, 32)])
def test_prompts(heads, q_heads, dim, page, dt):
    """Prompts from nothing and behind cached tokens, odd lengths, tiles cut everywhere."""
    run(heads, q_heads, dim, page, [200, 1, 65, 129, 0, 64], [200, 77, 65, 300, 5, 191], dt, seed=page + dim)


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("dt,out_dt", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("dim,window", [(64, 0), (80, 100), (128, 0), (256, 70), (48, 1)])
def test_many_rows(dim, page, dt, out_dt, window):
    """Prompts of the size that the prompt kernel takes, rows without keys and missing pages
    among them."""
    def edit(table, q_start, kv_len, ks, vs):
        table[1, 1] = -1
        kv_len[3] = 30                                   # 40 rows of 30 tokens
    run(16, 32, dim, page, [257, 65, 1, 40, 130], [300, 200, 250, 40, 130], dt, out_dt, window=window,
        seed=dim, edit=edit)
    run(8, 24, dim, page, [257, 1, 90], [700, 650, 400], dt, out_dt, window=window, seed=dim + 1)


@pytest.mark.parametrize("dim", [128, 80])
@pytest.mark.parametrize("page,out_dt", [(16, "bf16"), (128, "f32")])
def test_wide_prompts(dim, page, out_dt):
    """Enough bf16 columns for the workgroups of 256: whole, partly and barely filled, with
    step counts on every residue of the buffers, and windows."""
    news, lens = [130, 1, 40, 5], [130, 450, 300, 70]
    run(64, 128, dim, page, news, lens, "bf16", out_dt, seed=dim)
    run(86, 86, dim, page, [257, 20, 1], [257, 220, 129], "bf16", out_dt, seed=dim, window=65)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 200, 10 ** 9])
def test_windows(dt, window):
    run(2, 4, 64, 32, [1, 5, 150, 1], [400, 333, 301, 10], dt, window=window, seed=window % 97)


@pytest.mark.parametrize("dt,out_dt", [("bf16", "f32"), ("f32", "bf16")])
def test_mixed_types(dt, out_dt):
    run(2, 8, 128, 64, [1, 90, 4], [500, 130, 20], dt, out_dt)


# few heads: the decode kernel; many: the prompt kernel
BOTH = pytest.mark.parametrize("heads,q_heads", [(2, 4), (96, 192)])


@BOTH
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_sharp_and_flat_weights(dt, heads, q_heads):
    """Logits far apart (one key takes all), equal ones, and a negative scale."""
    run(heads, q_heads, 128, 64, [1, 1, 70], [300, 129, 200], dt, sharp=30.0)
    run(heads, q_heads, 128, 64, [1, 1, 70], [300, 129, 200], dt, sharp=0.0)
    run(heads, q_heads, 128, 64, [1, 1, 70], [300, 129, 200], dt, scale=-0.2)
    run(heads, q_heads, 128, 64, [1, 1, 70], [300, 129, 200], dt, sharp=1e-20)
    run(heads, q_heads, 128, 64, [1, 1, 70], [300, 129, 200], dt, scale=0.0)


@BOTH
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_large_queries(dt, heads, q_heads):
    """Queries near the type's end do not overflow on the way (their logits stay finite)."""
    run(heads, q_heads, 64, 16, [1, 60], [90, 77], dt, sharp=1e30, scale=1e-31)


@BOTH
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_page_scales_far_apart(dt, heads, q_heads):
    """Pages whose scales differ by many orders: a tiny one beside a large one."""
    def edit(table, q_start, kv_len, ks, vs):
        rng = np.random.default_rng(1)
        vs *= np.exp(rng.normal(0, 6, vs.shape)).astype(F32)
        ks *= np.exp(rng.normal(0, 1, ks.shape)).astype(F32)
    run(heads, q_heads, 64, 16, [1, 3, 100], [300, 50, 150], dt, edit=edit)


@BOTH
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_without_keys(dt, heads, q_heads):
    """More rows than tokens, no tokens at all, and rows behind the batch."""
    run(heads, q_heads, 64, 16, [5, 1, 80, 3], [3, 0, 20, 3], dt, tail=6)


@BOTH
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_bad_pages_are_not_seen(dt, heads, q_heads):
    def edit(table, q_start, kv_len, ks, vs):
        table[0, 1], table[0, 3] = -1, 1 << 30
        table[1, 0] = 10 ** 9                            # a sequence whose only page is missing
        table[2, :2] = -7
    run(heads, q_heads, 64, 16, [1, 1, 90, 3], [100, 9, 120, 40], dt, edit=edit)
    run(heads, q_heads, 64, 64, [1, 1, 90, 3], [300, 9, 190, 40], dt, edit=edit)


@BOTH
def test_bad_rows_and_lengths(heads, q_heads):
    def edit(table, q_start, kv_len, ks, vs):
        q_start[:] = [-4, 30, 1 << 30, 20]
        kv_len[:] = [40, -5, 1 << 30]
    run(heads, q_heads, 64, 16, [30, 1, 16], [40, 5, 16], edit=edit, max_new=30)


@BOTH
def test_bounds_of_the_batch(heads, q_heads):
    """Rows past max_new are left alone, tokens past max_len are not there."""
    run(heads, q_heads, 64, 16, [50, 1, 16], [60, 5, 16], max_new=29)
    run(heads, q_heads, 64, 16, [3, 1, 36], [40, 5, 36], max_len=30)


@BOTH
def test_strided_queries(heads, q_heads):
    run(heads, q_heads, 64, 16, [3, 1, 90], [40, 5, 100], strided=True)
    run(heads, q_heads, 80, 16, [3, 1, 90], [40, 5, 100], dt="f32", strided=True)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [1, 3])
def test_unaligned_queries(dt, shift):
    """Query rows aligned to their elements only."""
    q_start, kv_len, table, pages = seqs([2, 1, 90], [40, 5, 100], 16)
    k, v, ks, vs = cache(pages, 16, 16, 80, 3)
    c = N.KVCache(dev(k), dev(v), dev(ks), dev(vs))
    q = dev(np.random.default_rng(0).standard_normal((93, 64, 80)).astype(F32)).to(TYPES[dt])
    flat = torch.zeros(q.numel() + shift, dtype=q.dtype, device=DEV)
    flat[shift:] = q.reshape(-1)
    for most in (2, 90):      # both kernels (the rows past max_new are left alone)
        b = N.KVBatch(dev(table), dev(q_start), dev(kv_len), most, table.shape[1] * 16)
        outs = [torch.full((93, 64, 80), 7.0, dtype=q.dtype, device=DEV) for _ in range(2)]
        N.bitnet_attention(c, b, q, out=outs[0])
        N.bitnet_attention(c, b, flat[shift:].view(93, 64, 80), out=outs[1])
        assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 128), (256, 32)])
def test_captured_prompts(dim, page):
    """Prompts and drafted tokens in a graph, replayed over other lengths and queries with
    eager calls in between."""
    q_start, kv_len, table, pages = seqs([70, 3], [90, 200], page, width=32)
    k, v, ks, vs = cache(pages, 32, page, dim, 3)
    c = N.KVCache(dev(k), dev(v), dev(ks), dev(vs))
    qs, ln = dev(q_start), dev(kv_len)
    b = N.KVBatch(dev(table), qs, ln, 70, 32 * page)
    q = torch.zeros((73, 128, dim), dtype=torch.bfloat16, device=DEV)
    few = N.KVBatch(dev(table), dev(np.array([0, 1, 2], np.int32)), ln, 1, 32 * page)
    N.bitnet_attention(c, b, q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = N.bitnet_attention(c, b, q)
        one = N.bitnet_attention(c, few, q[:2])
    for n in range(4):
        q.normal_()
        ln.copy_(torch.tensor([90 - 7 * n, 200 - 31 * n], dtype=torch.int32))
        qs.copy_(torch.tensor([0, 70 - 20 * n, 73 - 20 * n], dtype=torch.int32))
        out.fill_(7.0)
        g.replay()
        want = torch.full_like(out, 7.0)
        N.bitnet_attention(c, b, q, out=want)
        assert torch.equal(out, want)
        assert torch.equal(one, N.bitnet_attention(c, few, q[:2]))


@BOTH
def test_shared_pages(heads, q_heads):
    """Two sequences on one prefix."""
    def edit(table, q_start, kv_len, ks, vs):
        table[1, :2] = table[0, :2]
    run(heads, q_heads, 64, 16, [1, 44, 1], [40, 60, 16], edit=edit)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("heads,q_heads,news,lens,page", [
    (1, 4, [1], [20011], 64), (2, 4, [1, 1, 2], [9001, 1, 5003], 16), (1, 1, [33], [7001], 128)])
def test_long_caches(dt, heads, q_heads, news, lens, page):
    """Few rows over many keys: the keys are split and joined."""
    run(heads, q_heads, 64, page, news, lens, dt, sharp=1.5)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_sizes_do_not_change_results_much(dt):
    """A loose max_len (a captured graph's) gives the same values within the bounds."""
    for max_len in (4096, 640, 64):
        q_start, kv_len, table, pages = seqs([1], [60], 64, width=64)
        k, v, ks, vs = cache(pages, 1, 64, 64, 3)
        c = N.KVCache(dev(k), dev(v), dev(ks), dev(vs))
        b = N.KVBatch(dev(table), dev(q_start), dev(kv_len), 1, max_len)
        q = np.random.default_rng(0).standard_normal((1, 4, 64)).astype(F32)
        qt = dev(q).to(TYPES[dt])
        out = N.bitnet_attention(c, b, qt)
        want, wl, absv, flat, top, reach = L.attention(k, v, ks, vs, table, q_start, kv_len,
                                                       qt.float().cpu().numpy(), 0.125, detail=True)
        tol, _ = attention_bounds(want, wl, absv, flat, top, reach, q, np.full(wl.shape, 60.0), dt == "f32")
        assert np.all(np.abs(host(out.float()) - want) <= tol)


def test_repeats_are_identical():
    """The same call twice gives the same bits (no order of arrival in any sum)."""
    q_start, kv_len, table, pages = seqs([1, 3, 70], [9000, 300, 500], 16)
    k, v, ks, vs = cache(pages, 2, 16, 128, 3)
    c = N.KVCache(dev(k), dev(v), dev(ks), dev(vs))
    b = N.KVBatch(dev(table), dev(q_start), dev(kv_len), 70, 9008)
    for heads in (8, 96):                             # both kernels
        q = dev(np.random.default_rng(0).standard_normal((74, heads, 128)).astype(F32))
        first = host(N.bitnet_attention(c, b, q))
        for _ in range(3):
            np.testing.assert_array_equal(host(N.bitnet_attention(c, b, q)), first)


def test_cache_beyond_4_gib():
    page, heads, dim = 128, 8, 256
    pages = (5 << 30) // (page * heads * dim)
    free, _ = torch.cuda.mem_get_info()
    if free < 14 << 30:
        pytest.skip("needs 14 GiB")
    big = N.KVCache.empty(pages, heads, page, dim, device=DEV)
    k, v, ks, vs = cache(2, heads, page, dim, 3)
    small = N.KVCache(dev(k), dev(v), dev(ks), dev(vs))
    for name in ("k", "v", "k_scale", "v_scale"):
        getattr(big, name)[pages - 1] = getattr(small, name)[0]
        getattr(big, name)[7] = getattr(small, name)[1]
    n, ln = dev(np.array([0, 1, 71], np.int32)), dev(np.array([200, 256], np.int32))
    q = dev(np.random.default_rng(0).standard_normal((71, 128, dim)).astype(F32))
    t0, t1 = np.array([[0, 1], [0, 1]], np.int32), np.array([[pages - 1, 7]] * 2, np.int32)
    for most in (70, 1):                              # both kernels
        out = [torch.zeros_like(q) for _ in range(2)]
        N.bitnet_attention(small, N.KVBatch(dev(t0), n, ln, most, 256), q, out=out[0])
        N.bitnet_attention(big, N.KVBatch(dev(t1), n, ln, most, 256), q, out=out[1])
        assert torch.equal(*out) and bool(out[0][0].any())
    del big
    torch.cuda.empty_cache()
