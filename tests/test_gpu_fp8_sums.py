"""Precision of the 8-bit path's products on the GPU.

The same token stands in every row and minus its output, rounded to fp16, is the bias: the output is then the
rest, rounded at 2^-11 of a rest that is itself 2^-11 of the sum, and shows the float32 sum's own error.
  exact products  (up to 16 tokens, or precise): the sums of the whole products, off by float32 additions
                  alone (oracle.accumulation_errors; the last rounding, 2^-22 of the sum at most, is added).
  8-bit products  the same about the sums of the products cut off as the 8-bit matrix instruction does.
"""

import numpy as np
import pytest
import torch

from oracle import fp8
from tests.test_fp8_sums_host import products, token_and_weights
from tests.test_gpu_fp8_precise import SHAPES, U, _dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("precise", [False, True])
@pytest.mark.parametrize("outliers", [False, True])
@pytest.mark.parametrize("K", [16, 128, 400, 1152])
@pytest.mark.parametrize("M,N", SHAPES)
def test_sums(kq, M, N, K, outliers, precise):
    xc, xs, wc, ws = token_and_weights(N, K, outliers, M + K)
    p = products(xc, xs, wc, ws)
    exact = p.sum(axis=1)
    bias = -torch.from_numpy(exact).to(torch.float16)
    y = kq.fp8_linear(*_dev(np.repeat(xc, M, axis=0), np.repeat(xs, M, axis=0)), *_dev(wc, ws), bias=bias.cuda(),
                      precise=precise)
    assert bool((y == y[:1]).all())                        # one token, one answer
    got = y[0].cpu().double().numpy() - bias.double().numpy()
    target = exact if precise or M <= 16 else fp8.cut_sums(xc[0], xs[0], wc, ws)
    # the output's own rounding and the sum's with the bias, taken off
    slack = 2.0 ** -11 * np.abs(got - exact) + (2.0 ** -22 + U) * np.abs(exact) + 2.0 ** -25
    err = got - target
    err = np.sign(err) * np.maximum(np.abs(err) - slack, 0.0)
    errors = fp8.accumulation_errors(target + err, target, p)
    assert not errors, errors


@pytest.mark.parametrize("K", [4096, 11008])
@pytest.mark.parametrize("M", [1, 20, 100])
def test_sums_long(kq, M, K):
    xc, xs, wc, ws = token_and_weights(272, K, True, K)
    p = products(xc, xs, wc, ws)
    bias = -torch.from_numpy(p.sum(axis=1)).to(torch.float16)
    for precise in (False, True):
        y = kq.fp8_linear(*_dev(np.repeat(xc, M, axis=0), np.repeat(xs, M, axis=0)), *_dev(wc, ws), bias=bias.cuda(),
                          precise=precise)
        got = y[0].cpu().double().numpy() - bias.double().numpy()
        target = p.sum(axis=1) if precise or M == 1 else fp8.cut_sums(xc[0], xs[0], wc, ws)
        errors = fp8.accumulation_errors(got, target, p)
        assert not errors, (precise, errors)
