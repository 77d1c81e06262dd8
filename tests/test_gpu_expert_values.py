"""Activations behind ternary products at the ends of the fp32 range, through the kernels for few and
for many rows."""

import numpy as np
import pytest
import torch

from oracle import bitnet_oracle as O
from oracle import experts_oracle as E
from ternary_weight_linear_bit_amd import _native as N

from experts_util import F32, dev, host

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
