"""Keys and values whose outputs nearly cancel, so that the rounding of a weight is not hidden by the output's own, and the
precision that the weights of the paged attention, and of attention with precise=True, have.

A weight p is multiplied as a sum of 16-bit numbers: the first is p rounded, so that what is left is at most half a step of
p, the next one that rounded, and so on: 2^-11 2^-11 with two of fp16, 2^-8 2^-8 2^-8 with three of bf16.  fp16 weights are
held at 2^6 of the largest or more, so half of fp16's smallest step, 2^-25, is at most 2^-31 of the largest weight."""

import numpy as np
import torch

from oracle import attention as oracle
from tests.attn_util import DT, quantized, widened

WEIGHT = {("fp16", "fp16"): (2.0 ** -22, 2.0 ** -31), ("bf16", "bf16"): (2.0 ** -24, 0.0),
          ("fp16", "fp8"): (2.0 ** -24, 0.0), ("bf16", "fp8"): (2.0 ** -24, 0.0)}
NUMBERS = {"fp16": 2, "bf16": 3, "fp8": 3}                  # of a weight, by the cache's type
KINDS = sorted(WEIGHT)


def rounded(x, dtype):
    return torch.from_numpy(np.asarray(x, np.float32)).to(DT[dtype])


def rows(n, Hkv, D, dtype, cache, seed):
    """n keys and values [n][Hkv][D] as 16-bit tensors (CPU): value 2 i + 1 is minus value 2 i, and its key nearly the same,
    so that the two weights differ by some percent and an output is some percent of its terms."""
    rng = np.random.default_rng(seed)
    k, v = rng.normal(size=(n, Hkv, D)), rng.normal(size=(n, Hkv, D))
    near = 0.03 if cache == "fp8" else 0.01
    k[1::2] = k[: n // 2 * 2: 2] + near * rng.normal(size=k[1::2].shape)
    v[1::2] = -v[: n // 2 * 2: 2]
    return rounded(k, dtype), rounded(v, dtype)


def cached(x, cache):
    """The float64 values that a cache holds of 16-bit rows."""
    x = x.double().numpy()
    return widened(*quantized(x)) if cache == "fp8" else x


def multiplied(q, K, V, scale, dtype, cache, numbers):
    """[n of q][D] float64: the sums with each weight as the sum of `numbers` 16-bit numbers, the rest in 64 bits."""
    kind, lift = ("fp16", 2.0 ** 6) if cache == "fp16" else ("bf16", 1.0)
    s = scale * (q @ K.T)
    p = np.exp(s - s.max(axis=1, keepdims=True)).astype(np.float32).astype(np.float64) * lift
    w, left = np.zeros_like(p), p
    for _ in range(numbers):
        part = rounded(left, kind).double().numpy()
        w, left = w + part, left - part
    return w @ V / p.sum(axis=1, keepdims=True)


def expect(q, K, V, scale, dtype, cache):
    return oracle.attend(q, K, V, scale, [len(K)] * len(q), *WEIGHT[dtype, cache])


def triples(B, dtype, seed):
    """B sequences of three keys and one query, rows of 32: [B][32], [B][3][32], [B][3][32] (CPU, 16-bit).  The first key
    has the largest weight and zeros for values; the others' weights lie between 0.2 and 0.8 of it and differ by 2^-12 to
    2^-11, with values of 1 and -1: an output is at most 2^-12, and what rounding leaves of the two weights stands beside it."""
    rng = np.random.default_rng(seed)
    q, k, v = np.zeros((B, 32)), np.zeros((B, 3, 32)), np.zeros((B, 3, 32))
    q[:, 0], q[:, 1] = 1.0, 2.0 ** -5
    k[:, 1:, 0] = -rng.integers(16, 96, size=(B, 1)) / 64.0
    k[:, 2, 1] = -rng.integers(8, 15, size=B) / 1024.0      # times 2^-5: 2^-12 to 2^-11
    v[:, 1], v[:, 2] = 1.0, -1.0
    return tuple(rounded(t, dtype) for t in (q, k, v))


def expect_triple(q, K, V):
    """As oracle.attend with scale 1, with what the two products of a score leave: one addition of half a step of a number up to
    1.5 (the products are exact), the scaling by log2 e (the factor's own rounding, the maximum's and the argument's), the
    exponential; three sums of three numbers."""
    u = 2.0 ** -24
    s = K @ q
    w = np.exp(s - s.max())
    rel = u * (np.abs(s).max() * 4 + 4) + 2.0 ** -24
    spread = w @ np.abs(V) / w.sum()
    return w @ V / w.sum(), (2 * rel + 6 * u) * spread
