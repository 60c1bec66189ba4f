"""GPU parity of attention where what a row sees is not finite at keys whose weights vanish."""

import numpy as np
import pytest

from oracle import attention as oracle
from tests.attn_util import WEIGHT, check, check_codes, dbl, heads

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64)])
@pytest.mark.parametrize("Tk", [600, 2000])                 # whole, and split over the keys
@pytest.mark.parametrize("low", [-300.0, float("-inf")])
def test_nan_of_no_weight(kq, dtype, D, Tk, low):
    """NaN among values that are seen reaches the output, however far below the largest its key's score is: whether
    the keys are split makes no difference."""
    Q, K, V = heads((4, 2, D), dtype, 1), heads((Tk, 1, D), dtype, 2), heads((Tk, 1, D), dtype, 3)
    Q[:, :, 0] = 1.0
    K[:, 0, 0] = 0.0
    K[:Tk // 2, 0, 0] = low                                 # weights of e^-300 are zero in float32, in 64 bits they add nothing
    V[70, 0, 5] = float("nan")
    assert (kq.attention_workspace_bytes(1, 4, Tk, False, 2, 1, D) > 0) == (Tk == 2000)
    o, tau = oracle.attention(dbl(Q), dbl(K)[Tk // 2:], dbl(V)[Tk // 2:], [0, 4], [0, Tk - Tk // 2], True, 1.0,
                              *WEIGHT[dtype, dtype])
    o[:, :, 5] = np.nan
    check(kq.attention(Q, K, V, scale=1.0), o, tau, dtype)
    if D == 128:
        check_codes(*kq.attention(Q, K, V, scale=1.0, fp8=True), o, tau)
