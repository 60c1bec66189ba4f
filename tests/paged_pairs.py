"""Cached keys and values whose outputs nearly cancel, so that the rounding of a weight is not hidden by the output's own,
and the precision that the paged attention's weights have.

A weight p is multiplied as hi + lo: hi is p rounded to 16 bits, so lo = p - hi is at most half a step of p, and lo rounded is
off by half a step of that: 2^-8 2^-8 (bf16), 2^-11 2^-11 (fp16).  fp16 weights are held at 2^6 of the largest or more, so
half of fp16's smallest step, 2^-25, is at most 2^-31 of the largest weight."""

import numpy as np
import torch

from oracle import attention as oracle
from tests.attn_util import DT, quantized, widened

WEIGHT = {("fp16", "fp16"): (2.0 ** -22, 2.0 ** -31), ("bf16", "bf16"): (2.0 ** -16, 0.0),
          ("fp16", "fp8"): (2.0 ** -16, 0.0), ("bf16", "fp8"): (2.0 ** -16, 0.0)}
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
    """[n of q][D] float64: the sums with each weight as the sum of `numbers` 16-bit numbers, all else exact."""
    kind, lift = ("fp16", 2.0 ** 6) if cache == "fp16" else ("bf16", 1.0)
    s = scale * (q @ K.T)
    p = np.exp(s - s.max(axis=1, keepdims=True)) * lift
    w, left = np.zeros_like(p), p
    for _ in range(numbers):
        part = rounded(left, kind).double().numpy()
        w, left = w + part, left - part
    return w @ V / p.sum(axis=1, keepdims=True)


def expect(q, K, V, scale, dtype, cache):
    return oracle.attend(q, K, V, scale, [len(K)] * len(q), *WEIGHT[dtype, cache])
