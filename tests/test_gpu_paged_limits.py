"""The largest batch of cached keys that a call takes."""

import numpy as np
import pytest
import torch

from oracle import attention as oracle
from tests.attn_util import WEIGHT, check, heads, on_gpu, quantized, widened

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,width", [(128, 65536), (127, 65536)])
def test_most_keys(kq, B, width):
    """2^37 keys in all, 2^31 blocks of 64, and a few less: each sequence has 2^30, nearly all of them at entries that
    name no page, and one page that is there (two sequences have two)."""
    page, D = 16384, 16
    rng = np.random.default_rng(1)
    k, v = rng.normal(size=(3, 1, page, D)), rng.normal(size=(3, 1, page, D))
    (ck, sk), (cv, sv) = quantized(k), quantized(v)
    table = np.full((B, width), -1, np.int32)
    there = [[int(rng.integers(3))] for _ in range(B)]
    there[0], there[-1] = [2, 0], [1, 2]
    for b, pages in enumerate(there):
        at = [0, width - 1] if len(pages) == 2 else [int(rng.integers(width))]
        table[b, at] = pages
    Q = heads((B, 2, D), "bf16", 2, 1.5)
    O = torch.full((B, 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    kq.paged_attention(Q, on_gpu(ck).view(torch.float8_e4m3fn), on_gpu(cv).view(torch.float8_e4m3fn), on_gpu(table),
                       on_gpu(np.full(B, 1 << 30, np.int32)), kscales=on_gpu(sk), vscales=on_gpu(sv), O=O)
    torch.cuda.synchronize()
    k64, v64 = widened(ck, sk), widened(cv, sv)
    q = Q.cpu().double().numpy()
    for b in (0, 1, B // 2, B - 2, B - 1):
        K, V = (np.concatenate([t[p, 0] for p in there[b]]) for t in (k64, v64))
        for h in range(2):
            o, tau = oracle.attend(q[b, h][None], K, V, D ** -0.5, [len(K)], *WEIGHT["bf16", "fp8"])
            check(O[b, h][None], o, tau, "bf16", f"sequence {b}")
    assert torch.isfinite(O).all() and (O != 7.0).all()
