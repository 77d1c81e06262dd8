"""bitnet_residual_norm on the GPU against the oracle, bit for bit."""

import numpy as np
import pytest
import torch

from oracle import bitnet_oracle as O
from oracle import layer_oracle as L
from ternary_weight_linear_bit_amd import _native as N
from ternary_weight_linear_bit_amd import inputs as I

from gpu_helpers import DEV, bf16_bits, dev, f32_bits, host

pytestmark = pytest.mark.gpu
F32 = np.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.lib()


def typed(x, dt):
    t = torch.from_numpy(np.ascontiguousarray(x, F32))
    t = t.to(torch.bfloat16) if dt == "bf16" else t
    return t.to(DEV), t.float().numpy()


def same(t, want, dt):
    if dt == "bf16":
        np.testing.assert_array_equal(bf16_bits(t), O.f32_to_bf16_bits(want))
    else:
        np.testing.assert_array_equal(f32_bits(host(t)), f32_bits(want))


def run(m, k, yd="bf16", hd="f32", ud="bf16", post=True, pre=True, gate="none", scale=0.3, eps=1e-5,
        in_place=False, quantize=True, offset=0, y=None, h=None, seed=0):
    rng = np.random.default_rng(300 + seed)
    y = rng.standard_normal((m, k)) if y is None else y
    h = 3 * rng.standard_normal((m, k)) if h is None else h

    def place(x, dt):
        t, f = typed(x, dt)
        if offset:
            flat = torch.zeros(t.numel() + offset, dtype=t.dtype, device=DEV)
            flat[offset:] = t.reshape(-1)
            t = flat[offset:].view(t.shape)
        return t, f
    yt, yf = place(y, yd)
    ht, hf = place(h, hd)
    g = {"none": None, "channel": rng.standard_normal(k), "token": rng.standard_normal((m, k))}[gate]
    gt, gf = (None, None) if g is None else place(g, yd)
    w1 = I.norm_weight(k, 1) if post else None
    w2 = I.norm_weight(k, 2) if pre else None
    ut = torch.full((m, k), 7.0, dtype=torch.bfloat16 if ud == "bf16" else torch.float32, device=DEV) if ud else None
    out, xq, xs = N.bitnet_residual_norm(yt, ht, h_out=ht if in_place else None, gate=gt, scale=scale, eps=eps,
                                         post_weight=None if w1 is None else dev(w1),
                                         pre_weight=None if w2 is None else dev(w2), u=ut, quantize=quantize)
    wh, wu, wq, ws = L.residual_norm(yf, hf, hd == "bf16", w1, gf, scale, w2, eps)
    assert (out is ht) == in_place
    same(out, wh, hd)
    if ud:
        same(ut, wu, ud)
    if quantize:
        np.testing.assert_array_equal(host(xq), wq)
        np.testing.assert_array_equal(f32_bits(host(xs)), f32_bits(ws))
    else:
        assert xq is None and xs is None


@pytest.mark.parametrize("k", [1, 7, 8, 64, 2047, 2048, 2560, 4100, 8192, 14336, 28672])
@pytest.mark.parametrize("yd", ["bf16", "f32"])
@pytest.mark.parametrize("hd", ["bf16", "f32"])
def test_widths(k, yd, hd):
    run(3, k, yd, hd, gate="channel", seed=k)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("pre", [True, False])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("in_place", [True, False])
def test_parts(post, pre, gate, in_place):
    for k in (2560, 333, 6912):
        run(5, k, "bf16", "bf16" if k == 333 else "f32", None, post, pre, gate, in_place=in_place, seed=k)


@pytest.mark.parametrize("quantize,ud", [(True, None), (False, "bf16"), (False, "f32"), (True, "f32"), (False, None)])
@pytest.mark.parametrize("k", [520, 5000, 11])
def test_outputs(quantize, ud, k):
    run(4, k, "f32", "bf16", ud, quantize=quantize, gate="token", in_place=True)
    run(4, k, "f32", "bf16", ud, quantize=quantize, gate="token", pre=False)


@pytest.mark.parametrize("m", [1, 2, 37, 700])
def test_tokens(m):
    run(m, 1000, gate="token", seed=m)
    run(m, 2560, "bf16", "bf16", seed=m)


@pytest.mark.parametrize("yd", ["bf16", "f32"])
def test_unaligned(yd):
    run(3, 264, yd, "f32", offset=1, gate="token")
    run(3, 8200, yd, "bf16", offset=3, gate="channel")


@pytest.mark.parametrize("eps", [0.0, 1e-5, 1.0])
def test_eps(eps):
    run(3, 640, eps=eps)


def test_means_at_rounding_borders():
    """Rows whose mean of squares lies on or next to a midpoint of two floats, where
    the float64 sum cannot decide (the exact sum has to), in both norms."""
    k = 64
    rows = np.zeros((4, k), F32)
    rows[0, 0], rows[0, 1] = 1 + 2.0 ** -12, 2.0 ** -40      # just above a midpoint
    rows[1, 0] = 1 + 2.0 ** -12                              # on it
    rows[2] = rows[0] * F32(2.0 ** 50)
    rows[3] = rows[0] * F32(2.0 ** -62)
    run(4, k, "f32", "f32", "f32", y=rows, h=np.zeros((4, k)), gate="none", scale=1.0, eps=0.0)
    run(4, k, "f32", "f32", "f32", y=np.zeros((4, k)), h=rows, post=False, scale=1.0, eps=0.0)
    # rows that do not fit in registers (groups read again)
    wide = np.zeros((2, 70000), F32)
    wide[:, 0], wide[:, 69999] = 1 + 2.0 ** -12, 2.0 ** -40
    run(2, 70000, "f32", "f32", "f32", y=np.zeros((2, 70000)), h=wide, post=False, scale=1.0, eps=1e-5)


def test_zero_and_large_rows():
    run(3, 256, "f32", "f32", "f32", y=np.zeros((3, 256)), h=np.zeros((3, 256)))
    run(3, 256, "f32", "f32", "f32", y=np.full((3, 256), 1e18), h=np.full((3, 256), -1e18), scale=1.0)


def test_stream_then_linear_like_the_prologue():
    """The codes are those that the act quantiser forms of h' with the same norm."""
    rng = np.random.default_rng(1)
    y, _ = typed(rng.standard_normal((6, 2560)), "bf16")
    h, _ = typed(rng.standard_normal((6, 2560)), "bf16")
    w = dev(I.norm_weight(2560, 3))
    h2, xq, xs = N.bitnet_residual_norm(y, h, pre_weight=w)
    wq, ws = N.bitnet_quantize_acts(h2, norm_weight=w)
    np.testing.assert_array_equal(host(xq), host(wq))
    np.testing.assert_array_equal(f32_bits(host(xs)), f32_bits(host(ws)))
