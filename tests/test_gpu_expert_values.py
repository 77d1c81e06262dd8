"""Activations behind ternary products at the ends of the fp32 range, through the kernels for few and
for many rows."""

import numpy as np
import pytest
import torch

from oracle import bitnet_oracle as O
from oracle import experts_oracle as E
from ternary_weight_linear_bit_amd import _native as N

from experts_util import F32, acts, assign, dev, host, matrices, routing
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

FEW, MANY = 64, 24064      # outputs: one block a workgroup, and more blocks than that kernel takes


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    N.lib()


def signs(n):
    """Weights with one +1 (even rows) or -1 (odd rows) a row, and their device matrix."""
    q = np.zeros((n, 64), np.int8)
    q[np.arange(n), np.arange(n) % 64] = 1 - 2 * (np.arange(n) % 2)
    return q, N.bitnet_repack_prefill(dev(O.pack_codes(q)))


def values(v, n, act):
    """act(v) in the even columns and act(-v) in the odd ones, [len(v), n]: codes of 1, scales v."""
    _, w = signs(n)
    x = np.ones((len(v), 64), np.int8)
    return host(N.bitnet_ternary_linear_act(w, dev(np.ones(1, F32)), n, dev(x), dev(np.asarray(v, F32)), act=act))


@pytest.mark.parametrize("n", [FEW, MANY])
def test_silu_of_large_values(n):
    """silu(v) is v and silu(-v) is -0 far beyond where e^-v is 0, up to the largest value; silu(+inf) is +inf
    and silu(-inf), -inf times 0, no number."""
    v = np.array([150, 2.0 ** 100, 2.3e38, 2.37e38, 2.5e38, 3e38, np.finfo(F32).max, np.inf], F32)
    y = values(v, n, "silu")
    np.testing.assert_array_equal(y[:, 0::2], np.repeat(v[:, None], n // 2, 1))
    assert (y[:-1, 1::2].view(np.uint32) == 0x80000000).all()
    assert np.isnan(y[-1, 1::2]).all()


@pytest.mark.parametrize("n", [FEW, MANY])
def test_silu_where_its_power_is_subnormal(n):
    """From -80 to -110 silu goes from 1.4e-33 to 0: within 2^-20 of its value and, where it is subnormal, a step
    of those, 2^-149 (two roundings), beside it."""
    v = np.r_[np.linspace(80, 110, 121), 87.0, 87.33, 87.34, 88.0, 91.0].astype(F32)
    y = values(v, n, "silu").astype(np.float64)
    z = v.astype(np.float64)[:, None]
    low, high = -z * np.exp(-z) / (1 + np.exp(-z)), z / (1 + np.exp(-z))
    assert (np.abs(y[:, 1::2] - low) <= 2.0 ** -20 * np.abs(low) + 2.0 ** -149).all()
    assert (np.abs(y[:, 0::2] - high) <= 2.0 ** -20 * high).all()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [FEW, MANY])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ["none", "relu2", "silu", "gelu"])
def test_no_number_stays_none(act, gated, n, dt):
    """A row whose scale is NaN and a column whose bias is NaN are NaN, and nothing else is; infinite biases
    give what the activation gives."""
    rng = np.random.default_rng(n)
    q, w = signs(n)
    x, d = rng.integers(-127, 128, (40, 64)).astype(np.int8), np.full(40, 0.01, F32)
    bias = rng.standard_normal(n).astype(F32)
    d[[3, 39]] = np.nan
    bias[[1, n - 1]] = np.nan
    bias[2], bias[4] = np.inf, -np.inf
    up = (w, torch.ones(1, device=DEV)) if gated else None
    ub = np.full(n, 5, F32)             # (u is not 0, so that infinities stay)
    args = dict(act=act, bias=dev(bias), up=up, up_bias=dev(ub) if gated else None, y_dtype=dt)
    y = host(N.bitnet_ternary_linear_act(w, dev(np.ones(1, F32)), n, dev(x), dev(d), **args).float())
    with np.errstate(all="ignore"):
        want, _ = E.product(q, F32(1), x, d, bias, act, (q, F32(1), ub) if gated else None)
    nan = np.zeros((40, n), bool)
    nan[[3, 39]] = nan[:, [1, n - 1]] = True
    nan[:, 4] |= act in ("silu", "gelu")             # -inf times 0
    np.testing.assert_array_equal(np.isnan(want), nan)
    np.testing.assert_array_equal(np.isnan(y), nan)
    inf = np.isinf(np.where(nan, 0, want))
    assert inf.any()
    np.testing.assert_array_equal(y[inf], want[inf])
    # (silu and gelu 2^-20 of the value and 2^-24 of |v| <= 6, times |u| <= 7; the last rounding 2^-8)
    rest = ~nan & ~inf
    np.testing.assert_allclose(y[rest], want[rest], rtol=2.0 ** -8 if dt is torch.bfloat16 else 2.0 ** -19,
                               atol=2.0 ** -18)


@pytest.mark.parametrize("n", [40, 6016])
def test_an_expert_whose_scale_is_no_number(n):
    """Its rows are NaN through each activation, the other experts' are as they were."""
    counts = [60, 50, 40]
    r, (first, _, _) = routing(assign(counts, 75, 2), 3)
    xq, d = acts(75, 128, 1)
    _, g, w = matrices(3, n, 128, 2)
    bad = N.TernaryExperts(w.w, dev(np.array([g[0], np.nan, g[2]], F32)), n, 128)
    for act in ("none", "relu2", "silu", "gelu"):
        want = host(N.bitnet_expert_linear(r, w, dev(xq), dev(d), act=act))
        y = host(N.bitnet_expert_linear(r, bad, dev(xq), dev(d), act=act))
        want[first[1]:first[2]] = np.nan
        np.testing.assert_array_equal(y, want)
