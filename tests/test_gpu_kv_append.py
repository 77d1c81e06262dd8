"""bitnet_kv_append on the GPU against the oracle, bit for bit: codes, scales, rotated
queries, and every byte that the call has to leave alone."""

import numpy as np
import pytest
import torch

from oracle import bitnet_oracle as O
from oracle import layer_oracle as L
from ternary_weight_linear_bit_amd import _native as N

from gpu_helpers import DEV, bf16_bits, dev, f32_bits, host
from layer_util import cache, seqs, tables

pytestmark = pytest.mark.gpu
F32 = np.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.lib()


def rounded(x, bf16):
    """(GPU tensor, fp32 values) of x in the call's type."""
    t = torch.from_numpy(np.ascontiguousarray(x, F32))
    t = t.to(torch.bfloat16) if bf16 else t
    return t.to(DEV), t.float().numpy()


def run(heads, q_heads, dim, page, news, lens, bf16, rot=None, inter=False, seed=0, strided=False,
        in_place=False, tail=0, edit=None, max_new=None, offset=0):
    rng = np.random.default_rng(100 + seed)
    q_start, kv_len, table, pages = seqs(news, lens, page, seed=seed)
    rot = dim if rot is None else rot
    T = int(q_start[-1]) + tail
    k, v, ks, vs = cache(pages, heads, page, dim, seed)
    if edit:
        edit(table, q_start, kv_len)
    table_rows = table.shape[1]
    cos, sin = tables(max(table_rows * page, 1), rot)
    x = rng.standard_normal((T, 2 * heads + q_heads, dim)) * np.exp(rng.normal(0, 1, (T, 1, 1)))
    if strided or offset:   # one fused projection: q, k and v lie side by side
        flat = torch.zeros(T * (2 * heads + q_heads) * dim + offset,
                           dtype=torch.bfloat16 if bf16 else torch.float32, device=DEV)
        xt, xf = rounded(x, bf16)
        flat[offset:] = xt.reshape(-1)
        xt = flat[offset:].view(T, 2 * heads + q_heads, dim)
        qt, kt, vt = xt[:, :q_heads], xt[:, q_heads:q_heads + heads], xt[:, q_heads + heads:]
        qf, kf, vf = xf[:, :q_heads], xf[:, q_heads:q_heads + heads], xf[:, q_heads + heads:]
    else:
        qt, qf = rounded(x[:, :q_heads], bf16)
        kt, kf = rounded(x[:, q_heads:q_heads + heads], bf16)
        vt, vf = rounded(x[:, q_heads + heads:], bf16)
    most = max(news) if max_new is None else max_new
    max_len = table_rows * page
    c = N.KVCache(dev(k), dev(v), dev(ks), dev(vs))
    b = N.KVBatch(dev(table), dev(q_start), dev(kv_len), most, max_len)
    out = qt if in_place else torch.full((T, q_heads, dim), 7.0, dtype=qt.dtype, device=DEV)
    kw = dict(cos=dev(cos), sin=dev(sin)) if rot else {}
    got = N.bitnet_kv_append(c, b, kt, vt, interleaved=inter, q=qt, q_out=out, **kw)
    assert got is out
    wk, wv, wks, wvs, wq = L.kv_append(k, v, ks, vs, table, q_start, kv_len, kf, vf,
                                       cos if rot else None, sin if rot else None, inter, qf, most, max_len)
    np.testing.assert_array_equal(f32_bits(host(c.k_scale)), f32_bits(wks))
    np.testing.assert_array_equal(f32_bits(host(c.v_scale)), f32_bits(wvs))
    np.testing.assert_array_equal(host(c.k), wk)
    np.testing.assert_array_equal(host(c.v), wv)
    kept = np.isnan(wq).all(-1)                        # rows outside every sequence
    wq = np.where(kept[..., None], qf if in_place else F32(7.0), wq)
    if bf16:
        np.testing.assert_array_equal(bf16_bits(out), O.f32_to_bf16_bits(wq))
    else:
        np.testing.assert_array_equal(f32_bits(host(out)), f32_bits(wq))


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("heads,q_heads,dim", [(5, 20, 128), (2, 2, 64), (1, 3, 16), (2, 4, 80), (1, 2, 256)])
def test_single_tokens(page, bf16, heads, q_heads, dim):
    lens = [1, 2, page - 1, page, page + 1, 3 * page + 5]
    run(heads, q_heads, dim, page, [1] * len(lens), lens, bf16, seed=page + dim)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("bf16,inter,rot", [(True, False, None), (False, True, None), (True, True, 32),
                                            (False, False, 24), (True, False, 6), (False, True, 10),
                                            (True, False, 0)])
def test_prompts(page, bf16, inter, rot):
    """Whole and partial prompts: starting, ending and both inside a page, idle sequences."""
    news = [page, 1, 2 * page + 3, 0, page - 1, 5, 3]
    lens = [page, 2 * page, 3 * page + 1, 7, 2 * page - 1, page + 2, 3]
    run(2, 4, 64, page, news, lens, bf16, rot=rot, inter=inter, seed=page)


@pytest.mark.parametrize("bf16", [True, False])
def test_fused_projection_rows(bf16):
    """Rows at a stride, 16-byte aligned and not."""
    run(2, 4, 64, 32, [5, 1, 40], [5, 17, 70], bf16, strided=True)
    run(2, 4, 64, 32, [5, 1, 40], [5, 17, 70], bf16, offset=1)
    run(1, 1, 48, 16, [5, 1, 40], [5, 17, 70], bf16, offset=3, rot=20, inter=True)


@pytest.mark.parametrize("bf16", [True, False])
def test_in_place_queries(bf16):
    run(2, 12, 128, 64, [3, 1, 9], [3, 66, 80], bf16, in_place=True, tail=2)
    run(1, 70, 80, 64, [3, 1, 9], [3, 66, 80], bf16, in_place=True, rot=40)


def test_rows_behind_the_batch_are_left():
    run(2, 4, 64, 32, [4, 1], [4, 33], True, tail=5)


def test_more_rows_than_tokens():
    """Rows with negative positions have no place; the rest goes where it belongs."""
    run(2, 4, 64, 16, [9, 20, 4], [5, 20, 0], False)


def test_bad_pages_and_lengths():
    """Page ids outside the cache, lengths and row numbers outside the batch."""
    def pages(table, q_start, kv_len):
        table[0, 1], table[1, 0], table[2, 0] = -5, 1 << 30, 10 ** 6
    run(2, 4, 64, 16, [30, 1, 16], [40, 5, 16], True, edit=pages)

    def rows(table, q_start, kv_len):
        q_start[:] = [0, 30, 1 << 30, 20]               # past the end, then back
        kv_len[:] = [40, 5, 1 << 30]
    run(2, 4, 64, 16, [30, 1, 16], [40, 5, 16], True, edit=rows, max_new=30)

    def negative(table, q_start, kv_len):
        q_start[:] = [-7, 3, 4, 20]
        kv_len[:] = [-3, 5, 16]
    run(2, 4, 64, 16, [30, 1, 16], [40, 5, 16], False, edit=negative)


def test_max_new_bounds_the_rows():
    run(2, 4, 64, 16, [30, 1, 16], [40, 5, 16], True, max_new=7)


@pytest.mark.parametrize("bf16", [True, False])
def test_token_by_token_like_the_oracle(bf16):
    """A sequence grown token by token: the scale only grows within a page, and every
    step requantises as the oracle does; a page used again starts anew."""
    rng = np.random.default_rng(4)
    page, heads, dim = 16, 2, 32
    k, v, ks, vs = cache(3, heads, page, dim, 1)
    ks[:], vs[:] = np.nan, np.nan                       # never written
    table = np.array([[2, 0, 2]], np.int32)             # the first page again for 32 ..
    c = N.KVCache(dev(k), dev(v), dev(ks), dev(vs))
    cos, sin = tables(48, dim)
    want = (k, v, ks, vs)
    for n in range(1, 40):
        x = rng.standard_normal((2, 1, heads, dim)) * (1 + (n % 7))
        kt, kf = rounded(x[0], bf16)
        vt, vf = rounded(x[1], bf16)
        b = N.KVBatch(dev(table), dev(np.array([0, 1], np.int32)), dev(np.array([n], np.int32)), 1, 48)
        N.bitnet_kv_append(c, b, kt, vt, cos=dev(cos), sin=dev(sin))
        *want, _ = L.kv_append(*want, table, np.array([0, 1]), np.array([n]), kf, vf, cos, sin)
        got = [host(c.k), host(c.v), host(c.k_scale), host(c.v_scale)]
        for g, w in zip(got, want):
            np.testing.assert_array_equal(g, w)


def test_extreme_rows():
    """Zeros (the scale's floor), sub-normals, the largest values, and a long page."""
    page, heads, dim = 128, 1, 16
    k, v, ks, vs = cache(2, heads, page, dim, 2)
    x = np.zeros((130, heads, dim), F32)
    x[1] = 2.0 ** -140
    x[2] = 3e38
    x[3] = -3e38
    x[128] = 1e-30
    table = np.array([[1, 0]], np.int32)
    c = N.KVCache(dev(k), dev(v), dev(ks), dev(vs))
    b = N.KVBatch(dev(table), dev(np.array([0, 130], np.int32)), dev(np.array([130], np.int32)), 130, 256)
    N.bitnet_kv_append(c, b, dev(x), dev(x[::-1].copy()))
    with np.errstate(under="ignore"):
        wk, wv, wks, wvs, _ = L.kv_append(k, v, ks, vs, table, np.array([0, 130]), np.array([130]), x,
                                          x[::-1])
    np.testing.assert_array_equal(host(c.k), wk)
    np.testing.assert_array_equal(host(c.v), wv)
    np.testing.assert_array_equal(f32_bits(host(c.k_scale)), f32_bits(wks))
    np.testing.assert_array_equal(f32_bits(host(c.v_scale)), f32_bits(wvs))


def test_cache_beyond_4_gib():
    """Pages whose byte offsets pass 2^32."""
    page, heads, dim = 128, 8, 256
    pages = (5 << 30) // (page * heads * dim)
    free, _ = torch.cuda.mem_get_info()
    if free < 14 << 30:
        pytest.skip("needs 14 GiB")
    c = N.KVCache.empty(pages, heads, page, dim, device=DEV)
    table = np.array([[pages - 1, 3]], np.int32)
    rng = np.random.default_rng(9)
    x = rng.standard_normal((130, heads, dim)).astype(F32)
    b = N.KVBatch(dev(table), dev(np.array([0, 130], np.int32)), dev(np.array([130], np.int32)), 130, 256)
    N.bitnet_kv_append(c, b, dev(x), dev(2 * x))
    # the same pages in a cache of two
    k, v, ks, vs = cache(2, heads, page, dim, 2)
    table2 = np.array([[0, 1]], np.int32)
    wk, wv, wks, wvs, _ = L.kv_append(k, v, ks, vs, table2, np.array([0, 130]), np.array([130]), x, 2 * x)
    np.testing.assert_array_equal(host(c.k[pages - 1]), wk[0])
    np.testing.assert_array_equal(host(c.v[pages - 1]), wv[0])
    np.testing.assert_array_equal(host(c.k[3, :, :2]), wk[1, :, :2])
    np.testing.assert_array_equal(host(c.v_scale[pages - 1]), wvs[0])
    del c
    torch.cuda.empty_cache()
