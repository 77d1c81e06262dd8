"""The binding of the cache, attention and residual calls: threads, and arguments that contradict
each other."""

import ctypes
import os
import threading

import pytest
import torch

from ternary_weight_linear_bit_amd import _native as N

from test_layer_abi import A, EALIGN, EWS, a_batch, a_cache, attend, batch, cpu, kv, z  # noqa: F401


def test_dtype_codes_are_seen_whole(monkeypatch):
    """A thread that asks for a dtype's code while another is making the table gets it."""
    real, half, go = N._dtype_code, threading.Event(), threading.Event()

    def slow(dtype):
        if threading.current_thread().name == "first" and dtype is torch.bfloat16:
            half.set()
            assert go.wait(20)
        return real(dtype)
    monkeypatch.setattr(N, "_codes", {})
    monkeypatch.setattr(N, "_dtype_code", slow)
    got = []
    t = threading.Thread(target=lambda: got.append(N._code(torch.float32, "q")), name="first")
    t.start()
    try:
        assert half.wait(20)
        assert N._code(torch.bfloat16, "q") == N.BITNET_BF16
    finally:
        go.set()
        t.join()
    assert got == [N.BITNET_F32] and N._code(torch.float32, "q") == N.BITNET_F32
    with pytest.raises(ValueError, match="q: expected"):
        N._code(torch.float16, "q")


def test_out_dtype_that_contradicts_out(cpu):   # noqa: F811
    q = z(4, 4, 32)
    for out, dtype in ((z(4, 4, 32), torch.bfloat16), (z(4, 4, 32, dtype=torch.bfloat16), torch.float32)):
        with pytest.raises(ValueError, match="out_dtype"):
            cpu.bitnet_attention(a_cache(cpu), a_batch(cpu), q, out=out, out_dtype=dtype)
        with pytest.raises(AssertionError, match="reached the C library"):      # the same one is fine
            cpu.bitnet_attention(a_cache(cpu), a_batch(cpu), q, out=out, out_dtype=out.dtype)


@pytest.mark.parametrize("shape", [
    dict(seqs=1, width=4096, tokens=1, max_new=1, max_len=200000),          # a token over a long cache
    dict(seqs=1, width=4096, tokens=200, max_new=200, max_len=200000)],     # a prompt's part over it
    ids=["decode", "prompt"])
def test_workspaces_that_do_not_suffice(shape):
    """Both kernels split the keys of such a call: none, a byte less and a misaligned workspace are
    refused before anything is launched."""
    if not os.path.exists(N.LIB_PATH):
        pytest.skip("libbitnet_mi355x.so not built")
    lib = N.lib()
    c, b = kv(), batch(**shape)
    need = lib.bitnet_attention_workspace_bytes(ctypes.byref(kv(k=None, v=None)), ctypes.byref(b), 4)
    assert need > 0 and need % ((128 + 4) * 4) == 0      # columns of head_dim + 4 floats
    assert attend(lib, c, b, ws=None) == EWS
    assert attend(lib, c, b, ws_bytes=need - 1) == EWS
    assert attend(lib, c, b, ws=A + 4, ws_bytes=need) == EALIGN
