"""The paged attention's tolerances, without a GPU: they take the weights' 16-bit numbers and refuse one number less."""

import numpy as np
import pytest

from oracle import fp8
from tests import paged_pairs as pairs
from tests.attn_util import check


@pytest.mark.parametrize("dtype,cache", pairs.KINDS)
@pytest.mark.parametrize("n,D", [(8, 128), (30, 64), (17, 128)])
def test_one_number_is_not_enough(dtype, cache, n, D):
    k, v = pairs.rows(n, 1, D, dtype, cache, n)
    K, V = (pairs.cached(t, cache)[:, 0] for t in (k, v))
    q = pairs.rounded(np.random.default_rng(1).normal(size=(4, D)), dtype).double().numpy()
    o, tau = pairs.expect(q, K, V, D ** -0.5, dtype, cache)
    all_, one = (pairs.multiplied(q, K, V, D ** -0.5, dtype, cache, m) for m in (pairs.NUMBERS[cache], 1))
    check(pairs.rounded(all_, dtype), o, tau, dtype)
    with pytest.raises(AssertionError, match="of the bound"):
        check(pairs.rounded(one, dtype), o, tau, dtype)


@pytest.mark.parametrize("dtype,cache", [kind for kind in pairs.KINDS if kind[1] != "fp16"])
def test_codes_of_one_number(dtype, cache):
    """(One fp16 number is within what codes allow: 30 weights' errors of 2^-12 add up to 4e-5 here, and the bound of
    float32 scores alone is 1e-4.)"""
    k, v = pairs.rows(30, 1, 128, dtype, cache, 5)
    K, V = (pairs.cached(t, cache)[:, 0] for t in (k, v))
    q = pairs.rounded(np.random.default_rng(2).normal(size=(16, 128)), dtype).double().numpy()
    o, tau = pairs.expect(q, K, V, 128 ** -0.5, dtype, cache)
    for m, good in ((pairs.NUMBERS[cache], True), (1, False)):
        codes, scales = fp8.quantize(pairs.multiplied(q, K, V, 128 ** -0.5, dtype, cache, m))
        assert (not fp8.check_codes(codes, scales, o, tau)) == good


@pytest.mark.parametrize("dtype,cache", pairs.KINDS)
def test_one_number_less(dtype, cache):
    q, k, v = pairs.triples(64, dtype, 3)
    far = 0
    for b in range(64):
        K, V = (pairs.cached(t[b], cache) for t in (k, v))
        qb = q[b].double().numpy()
        o, tau = pairs.expect_triple(qb, K, V)
        y = [pairs.multiplied(qb[None], K, V, 1.0, dtype, cache, pairs.NUMBERS[cache] - m)[0] for m in (0, 1)]
        check(pairs.rounded(y[0], dtype), o, tau, dtype)
        try:
            check(pairs.rounded(y[1], dtype), o, tau, dtype)
        except AssertionError:
            far += 1
    assert far > 8, far
