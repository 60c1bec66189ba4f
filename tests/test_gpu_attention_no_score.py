"""GPU parity of attention for rows none of whose scores is above minus infinity: zeros."""

import numpy as np
import pytest
import torch

from oracle import attention as oracle
from tests.attn_util import WEIGHT, Cache, check, check_codes, cumulative, dbl, heads, on_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n", [100, 2000])                  # whole, and split
def test_no_score_above_minus_infinity(kq, dtype, n):
    """Rows all of whose scores are minus infinity give zeros, whatever the values; the next sequence's are its own."""
    cu_q, cu_k = cumulative([3, 2]), cumulative([n, 30])
    Q, K, V = heads((5, 2, 128), dtype, 4), heads((n + 30, 1, 128), dtype, 5), heads((n + 30, 1, 128), dtype, 6)
    Q[:, :, 0] = 1.0
    K[:n, 0, 0] = float("-inf")
    V[n // 3, 0, 3], V[n // 2, 0, 4], V[n - 20, 0, 5] = float("inf"), float("nan"), float("-inf")
    o, tau = np.zeros((5, 2, 128)), np.zeros((5, 2, 128))
    o[3:], tau[3:] = oracle.attention(dbl(Q)[3:], dbl(K)[n:], dbl(V)[n:], [0, 2], [0, 30], True,
                                      float(np.float32(128 ** -0.5)), *WEIGHT[dtype, dtype])
    check(kq.attention(Q, K, V, on_gpu(cu_q), on_gpu(cu_k)), o, tau, dtype)
    check_codes(*kq.attention(Q, K, V, on_gpu(cu_q), on_gpu(cu_k), fp8=True), o, tau)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("lengths", [[100, 30], [3000, 30]])
def test_no_score_above_minus_infinity_paged(kq, dtype, lengths):
    c = Cache(lengths, 1, 128, 16, dtype, dtype, 7)
    Q = heads((2, 2, 128), dtype, 8)
    Q[:, :, 0] = 1.0
    pages = torch.from_numpy(c.table[0][: -(-lengths[0] // 16)].astype(np.int64)).cuda()
    c.k[pages, :, :, 0] = float("-inf")
    for j, value in ((3, "inf"), (lengths[0] // 2, "nan"), (lengths[0] - 1, "-inf")):
        c.v[int(c.table[0, j // 16]), 0, j % 16, j % 7] = float(value)
    c.k64, c.v64 = dbl(c.k), dbl(c.v)
    with np.errstate(invalid="ignore"):
        o, tau = oracle.paged(dbl(Q), c.k64, c.v64, c.table, c.lengths, float(np.float32(128 ** -0.5)), *WEIGHT[dtype, dtype])
    o[0] = tau[0] = 0.0
    check(kq.paged_attention(Q, *c.args()), o, tau, dtype)
    check_codes(*kq.paged_attention(Q, *c.args(), fp8=True), o, tau)
