"""Refusals of the cache, attention and residual calls: the C ABI rejects bad
arguments before any HIP call, the binding rejects bad tensors before the C call."""

import ctypes
import os

import pytest
import torch

from ternary_weight_linear_bit_amd import _native as N

OK, ENULL, ESHAPE, EDTYPE, EALIGN, EWS = 0, 1, 2, 3, 4, 5
A = 0x10000        # never dereferenced: every call below fails validation


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(N.LIB_PATH):
        pytest.skip("libbitnet_mi355x.so not built")
    return N.lib()


def kv(**kw):
    f = dict(k=A, v=A, k_scale=A, v_scale=A, pages=8, kv_heads=2, page=64, head_dim=128)
    f.update(kw)
    return N.BitnetKvCache(*f.values())


def batch(**kw):
    f = dict(table=A, q_start=A, kv_len=A, seqs=3, width=4, tokens=5, max_new=2, max_len=200)
    f.update(kw)
    return N.BitnetKvBatch(*f.values())


def rows(**kw):
    f = dict(k=A, v=A, q=A, q_out=A, k_stride=256, v_stride=256, q_stride=512, dtype=0, q_heads=4,
             cos=A, sin=A, positions=200, rotary=128, interleaved=0)
    f.update(kw)
    return N.BitnetKvRows(*f.values())


BAD_CACHE = [(dict(page=48), ESHAPE), (dict(page=0), ESHAPE), (dict(head_dim=24), ESHAPE),
             (dict(head_dim=272), ESHAPE), (dict(head_dim=0), ESHAPE), (dict(kv_heads=0), ESHAPE),
             (dict(kv_heads=65536), ESHAPE), (dict(pages=0), ESHAPE), (dict(pages=1 << 31), ESHAPE),
             (dict(k=None), ENULL), (dict(v_scale=None), ENULL), (dict(k=A + 8), EALIGN),
             (dict(v=A + 4), EALIGN), (dict(k_scale=A + 2), EALIGN)]
BAD_BATCH = [(dict(seqs=-1), ESHAPE), (dict(seqs=65536), ESHAPE), (dict(width=0), ESHAPE),
             (dict(width=1 << 25), ESHAPE), (dict(tokens=-1), ESHAPE), (dict(tokens=1 << 31), ESHAPE),
             (dict(max_new=0), ESHAPE), (dict(max_new=6), ESHAPE), (dict(max_len=-1), ESHAPE),
             (dict(max_len=257), ESHAPE), (dict(table=None), ENULL), (dict(q_start=None), ENULL),
             (dict(kv_len=None), ENULL), (dict(table=A + 2), EALIGN)]


@pytest.mark.parametrize("bad,want", BAD_CACHE)
def test_cache_refusals(lib, bad, want):
    c, b, r = kv(**bad), batch(), rows()
    assert lib.bitnet_kv_append(ctypes.byref(c), ctypes.byref(b), ctypes.byref(r), None) == want
    assert attend(lib, c, b) == want


@pytest.mark.parametrize("bad,want", BAD_BATCH)
def test_batch_refusals(lib, bad, want):
    c, b, r = kv(), batch(**bad), rows()
    assert lib.bitnet_kv_append(ctypes.byref(c), ctypes.byref(b), ctypes.byref(r), None) == want
    assert attend(lib, c, b) == want


@pytest.mark.parametrize("bad,want", [
    (dict(dtype=2), EDTYPE), (dict(rotary=130), ESHAPE), (dict(rotary=7), ESHAPE),
    (dict(rotary=-2), ESHAPE), (dict(interleaved=2), ESHAPE), (dict(q_heads=3), ESHAPE),
    (dict(q_heads=0), ESHAPE), (dict(k_stride=255), ESHAPE), (dict(v_stride=0), ESHAPE),
    (dict(q_stride=511), ESHAPE), (dict(positions=199), ESHAPE), (dict(k=None), ENULL),
    (dict(v=None), ENULL), (dict(q_out=None), ENULL), (dict(cos=None), ENULL),
    (dict(q_stride=640), ESHAPE),          # in place needs contiguous queries
    (dict(k=A + 2), EALIGN), (dict(q=A + 32 + 2, q_out=A), EALIGN), (dict(q=A + 64, q_out=A + 4), EALIGN),
    (dict(sin=A + 1), EALIGN)])
def test_append_refusals(lib, bad, want):
    c, b, r = kv(), batch(), rows(**bad)
    assert lib.bitnet_kv_append(ctypes.byref(c), ctypes.byref(b), ctypes.byref(r), None) == want


def attend(lib, c, b, q=A, q_dtype=0, q_stride=512, q_heads=4, scale=1.0, window=0, out=A,
           out_dtype=0, lse=A, ws=A, ws_bytes=1 << 40):
    return lib.bitnet_attention(ctypes.byref(c), ctypes.byref(b), q, q_dtype, q_stride, q_heads, scale,
                                window, out, out_dtype, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("bad,want", [
    (dict(q_dtype=3), EDTYPE), (dict(out_dtype=-1), EDTYPE), (dict(q_heads=5), ESHAPE),
    (dict(q_heads=0), ESHAPE), (dict(q_stride=511), ESHAPE), (dict(window=-1), ESHAPE),
    (dict(scale=float("nan")), ESHAPE), (dict(scale=float("inf")), ESHAPE), (dict(q=None), ENULL),
    (dict(out=None), ENULL), (dict(q=A + 2), EALIGN), (dict(out=A + 2), EALIGN),
    (dict(out_dtype=1, out=A + 1), EALIGN), (dict(out=A + 8), EALIGN), (dict(lse=A + 2), EALIGN)])
def test_attention_refusals(lib, bad, want):
    assert attend(lib, kv(), batch(), **bad) == want


def test_attention_workspace(lib):
    f = lib.bitnet_attention_workspace_bytes
    c, b = kv(k=None, v=None), batch(table=None)     # sizes alone count
    for bad in (kv(page=5), kv(head_dim=8)):
        assert f(ctypes.byref(bad), ctypes.byref(b), 4) == 0
    assert f(None, ctypes.byref(b), 4) == 0 and f(ctypes.byref(c), ctypes.byref(b), 3) == 0
    assert f(ctypes.byref(c), ctypes.byref(batch(seqs=0)), 4) == 0
    # few rows over a long cache are split; the halves need a place
    long = batch(width=4096, max_len=200000, seqs=1, tokens=1, max_new=1)
    need = f(ctypes.byref(c), ctypes.byref(long), 4)
    if need:
        assert attend(lib, kv(), long, ws=None) == EWS
        assert attend(lib, kv(), long, ws_bytes=need - 1) == EWS
        assert attend(lib, kv(), long, ws=A + 4, ws_bytes=need) == EALIGN


def test_launches_beyond_the_runtime(lib):
    """Sizes whose grids the runtime cannot count are refused, not passed to it."""
    c, r = kv(page=128), rows(positions=1 << 30)
    big = batch(seqs=65535, width=1 << 20, tokens=1 << 30, max_new=1 << 20, max_len=1 << 27)
    assert lib.bitnet_kv_append(ctypes.byref(c), ctypes.byref(big), ctypes.byref(r), None) == ESHAPE
    assert attend(lib, c, big) == ESHAPE
    assert lib.bitnet_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(big), 4) == 0
    wide = batch(seqs=1, tokens=1 << 30, max_new=1 << 30)
    assert attend(lib, kv(kv_heads=1), wide, q_heads=64, q_stride=64 * 128) == ESHAPE
    assert lib.bitnet_residual_norm(ctypes.byref(res(M=1 << 22)), None) == ESHAPE


def test_nothing_to_do(lib):
    for b in (batch(seqs=0, table=None, q_start=None, kv_len=None), batch(tokens=0, max_new=1)):
        c, r = kv(k=None), rows(k=None, q=None)
        assert lib.bitnet_kv_append(ctypes.byref(c), ctypes.byref(b), ctypes.byref(r), None) == OK
        assert attend(lib, c, b, q=None, out=None, ws=None, ws_bytes=0) == OK
    assert lib.bitnet_kv_append(None, ctypes.byref(batch()), ctypes.byref(rows()), None) == ENULL
    assert lib.bitnet_attention(None, ctypes.byref(batch()), A, 0, 512, 4, 1.0, 0, A, 0, None, None, 0,
                                None) == ENULL


def res(**kw):
    f = dict(y=A, h=A, gate=A, h_out=A, u=A, post_weight=A, pre_weight=A, x_q=A, x_scale=A, M=3, K=40,
             gate_stride=40, y_dtype=0, h_dtype=1, u_dtype=1, scale=1.0, eps=1e-5)
    f.update(kw)
    return N.BitnetResidual(*f.values())


@pytest.mark.parametrize("bad,want", [
    (dict(y_dtype=2), EDTYPE), (dict(h_dtype=2), EDTYPE), (dict(u_dtype=2), EDTYPE), (dict(M=-1), ESHAPE),
    (dict(M=1 << 31), ESHAPE), (dict(K=0), ESHAPE), (dict(K=1 << 31), ESHAPE), (dict(gate_stride=39), ESHAPE),
    (dict(scale=float("inf")), ESHAPE), (dict(eps=-1.0), ESHAPE), (dict(eps=float("nan")), ESHAPE),
    (dict(y=None), ENULL), (dict(h=None), ENULL), (dict(h_out=None), ENULL), (dict(x_q=None), ENULL),
    (dict(x_scale=None), ENULL), (dict(y=A + 2), EALIGN), (dict(h=A + 1), EALIGN), (dict(gate=A + 2), EALIGN),
    (dict(u=A + 1), EALIGN), (dict(pre_weight=A + 2), EALIGN), (dict(x_scale=A + 2), EALIGN)])
def test_residual_refusals(lib, bad, want):
    r = res(**bad)
    assert lib.bitnet_residual_norm(ctypes.byref(r), None) == want


def test_residual_nothing_to_do(lib):
    assert lib.bitnet_residual_norm(ctypes.byref(res(M=0, y=None, h=None)), None) == OK
    assert lib.bitnet_residual_norm(None, None) == ENULL


def test_packed_structs_match_the_header():
    """The binding packs two structs itself: the same bytes as their ctypes classes."""
    assert N._ROWS.size == ctypes.sizeof(N.BitnetKvRows)
    v = (1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14)
    assert N._ROWS.pack(*v) == bytes(N.BitnetKvRows(*v))
    assert N._RESIDUAL.size == ctypes.sizeof(N.BitnetResidual)
    v = (1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 0.5, 0.25)
    assert N._RESIDUAL.pack(*v) == bytes(N.BitnetResidual(*v))


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------

class _NoCall:
    def __getattr__(self, name):
        if name.endswith("_workspace_bytes"):
            return lambda *a: 0

        def call(*a):
            raise AssertionError(f"{name} reached the C library with a bad tensor")
        return call


class _Here:
    """Stands for a CUDA tensor's device check and the stream."""
    def __init__(self, device, stream):
        pass

    def __enter__(self):
        return None

    def __exit__(self, *exc):
        pass


@pytest.fixture
def cpu(monkeypatch):
    monkeypatch.setattr(N, "_need_cuda", lambda *ts: None)
    monkeypatch.setattr(N, "lib", lambda: _NoCall())
    monkeypatch.setattr(N, "_On", _Here)
    real = N._rows

    def rows_of(t, heads, dim, name):
        class T:   # a CPU tensor that says it is a CUDA one
            is_cuda = True

            def __getattr__(self, a):
                return getattr(t, a)
        return real(T(), heads, dim, name)
    monkeypatch.setattr(N, "_rows", rows_of)
    return N


def z(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def a_cache(n, heads=2, page=16, dim=32):
    return n.KVCache(z(3, heads, page, dim, dtype=torch.int8), z(3, heads, dim, page, dtype=torch.int8),
                     z(3, heads), z(3, heads))


def a_batch(n):
    return n.KVBatch(z(2, 2, dtype=torch.int32), z(3, dtype=torch.int32), z(2, dtype=torch.int32), 2, 30)


def test_binding_rejects_bad_caches(cpu):
    i8 = torch.int8
    k, v, s = z(3, 2, 16, 32, dtype=i8), z(3, 2, 32, 16, dtype=i8), z(3, 2)
    for args in ((k, k, s, s), (k, v, s, z(3, 1)), (k.float(), v, s, s), (k, v, s.double(), s), (k[0], v, s, s),
                 (z(3, 2, 24, 32, dtype=i8), z(3, 2, 32, 24, dtype=i8), s, s),
                 (z(3, 2, 16, 24, dtype=i8), z(3, 2, 24, 16, dtype=i8), s, s)):
        with pytest.raises(ValueError):
            cpu.KVCache(*args)
    i32 = torch.int32
    for args in ((z(2, 2), z(3, dtype=i32), z(2, dtype=i32), 1, 1),
                 (z(2, 2, dtype=i32), z(2, dtype=i32), z(2, dtype=i32), 1, 1),
                 (z(2, 2, dtype=i32), z(3, dtype=i32), z(3, dtype=i32), 1, 1),
                 (z(2, 2, dtype=i32), z(3, dtype=i32), z(2, dtype=i32), 0, 1),
                 (z(2, dtype=i32), z(3, dtype=i32), z(2, dtype=i32), 1, 1)):
        with pytest.raises(ValueError):
            cpu.KVBatch(*args)


@pytest.mark.parametrize("bad", [
    dict(k=z(4, 3, 32)), dict(k=z(4, 2, 16)), dict(v=z(5, 2, 32)), dict(v=z(4, 2, 32, dtype=torch.bfloat16)),
    dict(k=z(4, 32, 2).transpose(1, 2)), dict(cos=z(30, 16)), dict(cos=z(30, 16), sin=z(30, 8)),
    dict(cos=z(30, 16).double(), sin=z(30, 16).double()), dict(q=z(4, 4, 16)), dict(q=z(3, 4, 32)),
    dict(q=z(4, 4, 32).double()), dict(q=z(4, 4, 32), q_out=z(4, 2, 32)), dict(q_out=z(4, 4, 32))])
def test_binding_rejects_bad_rows(cpu, bad):
    args = dict(k=z(4, 2, 32), v=z(4, 2, 32))
    args.update(bad)
    with pytest.raises(ValueError):
        cpu.bitnet_kv_append(a_cache(cpu), a_batch(cpu), **args)


@pytest.mark.parametrize("bad", [
    dict(q=z(4, 3, 32)), dict(q=z(4, 4, 16)), dict(out=z(4, 4, 16)), dict(out=z(4, 4, 32).double()),
    dict(lse=z(4, 2)), dict(lse=z(4, 4).double()), dict(q=z(4, 4, 64)[..., ::2])])
def test_binding_rejects_bad_queries(cpu, bad):
    args = dict(q=z(4, 4, 32))
    args.update(bad)
    with pytest.raises(ValueError):
        cpu.bitnet_attention(a_cache(cpu), a_batch(cpu), **args)


@pytest.mark.parametrize("bad", [
    dict(h=z(3, 8)), dict(y=z(4, 8).double()), dict(y=z(32)), dict(post_weight=z(7)),
    dict(pre_weight=z(8, dtype=torch.bfloat16)), dict(gate=z(7)), dict(gate=z(3, 8)),
    dict(gate=z(8, dtype=torch.bfloat16)), dict(h_out=z(4, 8, dtype=torch.bfloat16)), dict(u=z(4, 7)),
    dict(x_q=z(4, 8)), dict(x_scale=z(3)), dict(quantize=False, x_scale=z(4))])
def test_binding_rejects_bad_residuals(cpu, bad):
    args = dict(y=z(4, 8), h=z(4, 8))
    args.update(bad)
    with pytest.raises(ValueError):
        cpu.bitnet_residual_norm(**args)


def test_binding_rejects_other_devices():
    with pytest.raises(ValueError):
        N._one_device(z(1), None, torch.zeros(1, device="meta"))
    assert N._one_device(None, z(1)) == torch.device("cpu")

    class Stream:
        device = torch.device("cuda", 1)
    with pytest.raises(ValueError):
        N._On(torch.device("cuda", 0), Stream())
    with pytest.raises(ValueError):                  # host memory is no argument of a kernel
        N.bitnet_residual_norm(z(4, 8), z(4, 8))


@pytest.mark.parametrize("name", ["KVCache", "KVBatch"])
def test_attributes_are_fixed(name):
    # the C struct is made once, so an assignment could only be ignored
    c = getattr(N, name)
    x = c.__new__(c)
    x.max_len = x.k = 1
    for a in ("max_len", "k"):
        with pytest.raises(AttributeError, match="fixed"):
            setattr(x, a, 2)
        assert getattr(x, a) == 1
    x._struct = (1, None)
    x._struct = (2, None)
