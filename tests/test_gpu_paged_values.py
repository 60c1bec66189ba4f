"""GPU parity of the paged cache's attention where values are not finite, against the float64 oracle."""

import numpy as np
import pytest
import torch

from oracle import attention as oracle
from tests.attn_util import WEIGHT, Cache, check, check_codes, dbl, heads

pytestmark = pytest.mark.gpu

# lengths, table width (None: as wide as the longest needs): four wavefronts a head, two a head, dealt to runs that a second
# kernel joins 16 rows at a time, and by four heads
FORMS = {
    "whole": ([50, 40, 0, 129], None),
    "whole, many": ([int(n) for n in np.random.default_rng(0).integers(1, 90, size=300)], None),
    "dealt": ([5000, 700], None),
    "dealt, many": ([int(n) for n in np.random.default_rng(1).integers(30, 400, size=40)] + [3000], None),
}


def _expect(Q, c, dtype, cache):
    with np.errstate(invalid="ignore"):
        return oracle.paged(dbl(Q), c.k64, c.v64, c.table, c.lengths, float(np.float32(Q.shape[2] ** -0.5)), *WEIGHT[dtype, cache])


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(4, 1, 128, "bf16"), (8, 4, 64, "fp16"), (20, 1, 72, "bf16"), (4, 4, 128, "fp16")])
def test_infinities_that_are_seen(kq, form, Hq, Hkv, D, dtype):
    """A value of plus or minus infinity makes the outputs of its column that infinity, whatever its weight's
    rounding; both make NaN; other columns and heads keep their numbers."""
    lengths, width = FORMS[form]
    c = Cache(lengths, Hkv, D, 16, dtype, dtype, 90, width=width)
    rng = np.random.default_rng(91)

    def put(b, j, column, value):
        c.v[int(c.table[b, j // 16]), rng.integers(Hkv), j % 16, column] = value
    inf = float("inf")
    for b, n in enumerate(lengths):
        if n == 0 or b % 3 == 2:
            continue
        for column, values in ((1, [inf]), (2, [-inf]), (3, [inf, inf]), (4, [inf, -inf]), (6, [-inf, -inf, -inf])):
            for value in values:
                put(b, int(rng.integers(n)), column, value)
    c.v64 = dbl(c.v)
    Q = heads((len(lengths), Hq, D), dtype, 92, 1.5)
    o, tau = _expect(Q, c, dtype, dtype)
    assert np.isposinf(o).any() and np.isneginf(o).any() and np.isfinite(o[:, :, 0]).all()
    check(kq.paged_attention(Q, *c.args()), o, tau, dtype)
    if D == 128:
        check_codes(*kq.paged_attention(Q, *c.args(), fp8=True), o, tau)


@pytest.mark.parametrize("n", [1, 40, 640, 5000])
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp8")])
def test_nan_and_infinity_at_every_weight(kq, n, dtype, cache):
    """One key's values are not finite, for the key of the largest weight, of the smallest, and one between."""
    c = Cache([n] * 3, 1, 64, 16, dtype, cache, 93)
    q = heads((1, 1, 64), dtype, 94, 1.5)
    for b in range(3):
        K, _ = oracle.gather(c.k64, c.table[b], n, 16)
        order = np.argsort(K[:, 0] @ dbl(q)[0, 0])
        j = int(order[[-1, 0, n // 2][b]])
        at = int(c.table[b, j // 16]), 0, j % 16
        if cache == "fp8":
            c.v.view(torch.uint8)[at + (7,)] = 0xFF
            c.v64[at + (7,)] = np.nan
        else:
            c.v[at + (7,)], c.v[at + (8,)] = float("nan"), float("-inf")
            c.v64 = dbl(c.v)
    Q = q.expand(3, 1, 64).contiguous()
    o, tau = _expect(Q, c, dtype, cache)
    assert np.isnan(o[:, 0, 7]).all() and (cache == "fp8" or np.isneginf(o[:, 0, 8]).all())
    check(kq.paged_attention(Q, *c.args(), **c.scales()), o, tau, dtype)
