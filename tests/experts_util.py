"""Inputs shared by the tests of routing, experts' products and combination."""

import numpy as np
import torch

from oracle import bitnet_oracle as O
from oracle import experts_oracle as E
from ternary_weight_linear_bit_amd import _native as N
from ternary_weight_linear_bit_amd import inputs as I

from gpu_helpers import DEV, bf16_bits, dev, f32_bits, host

F32 = np.float32
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


def typed(x, dt):
    """(tensor on the GPU, fp32 numpy copy of its values)."""
    t = torch.from_numpy(np.ascontiguousarray(x, F32)).to(TORCH[dt])
    return t.to(DEV), t.float().numpy()


def assign(counts, tokens, topk, seed=0):
    """expert [tokens, topk] with these rows of each expert, in random order; -1 for the rest."""
    flat = np.full(tokens * topk, -1, np.int32)
    ids = np.repeat(np.arange(len(counts)), counts)
    flat[:ids.size] = ids
    return np.random.default_rng(seed).permutation(flat).reshape(tokens, topk)


def routing(expert, experts, weight=None, seed=0):
    """A Routing on the GPU made by the oracle, and its arrays (offset, pair, slot)."""
    expert = np.asarray(expert, np.int32)
    plan = E.plan(expert, experts)
    if weight is None:
        weight = np.random.default_rng(seed).uniform(0, 1, expert.shape).astype(F32)
    return N.Routing(dev(expert), dev(np.asarray(weight, F32)), *map(dev, plan)), plan


def acts(rows, k, seed):
    """Codes over the whole int8 range, -128 among them, and scales."""
    rng = np.random.default_rng(900 + seed)
    x = rng.integers(-128, 128, (rows, k)).astype(np.int8)
    return x, np.exp(rng.normal(0, 0.5, rows)).astype(F32) * F32(0.02)


def matrices(experts, n, k, seed):
    """(q [experts, N, K], scales) and their TernaryExperts."""
    q = np.stack([I.ternary_codes(n, k, 50 * seed + e) for e in range(experts)])
    scale = (0.02 * (1 + np.random.default_rng(seed).random(experts))).astype(F32)
    packed = np.stack([O.pack_codes(m) for m in q])
    return q, scale, N.TernaryExperts.from_packed(dev(packed), dev(scale))


def same(t, want, dt):
    """Bit for bit: tensor t of type dt against fp32 values before the last rounding."""
    if dt == "bf16":
        np.testing.assert_array_equal(bf16_bits(t), O.f32_to_bf16_bits(want))
    else:
        np.testing.assert_array_equal(f32_bits(host(t)), f32_bits(want))


def close(t, want, tol, dt):
    """Within tol, and the last rounding of bf16: half a step, 2^-8 of the value."""
    got = t.float().cpu().numpy().astype(np.float64)
    if dt == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) / tol))
