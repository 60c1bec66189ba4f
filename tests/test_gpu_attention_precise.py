"""GPU parity of attention with precise weights (several 16-bit numbers each) against the float64 oracle, at the tolerance of
the paged attention's weights (tests/paged_pairs.py, whose test without a GPU shows that one number less does not meet it)."""

import numpy as np
import pytest
import torch

from oracle import attention as oracle
from tests import paged_pairs as pairs
from tests.attn_util import check, check_codes, cumulative, dbl, heads, on_gpu, raw

pytestmark = pytest.mark.gpu


def _expect(Q, K, V, cq, ck, causal, dtype, scale=None):
    scale = Q.shape[2] ** -0.5 if scale is None else scale
    return oracle.attention(dbl(Q), dbl(K), dbl(V), cq, ck, causal, float(np.float32(scale)), *pairs.WEIGHT[dtype, dtype])


@pytest.mark.parametrize("lengths,past", [([5, 0, 131, 1, 257, 64], None), ([70, 3, 129], [20, 300, 1]), ([40, 1, 130], [200, 77, 131]),
                                          ([3, 0, 20, 1, 70], [1500, 40, 700, 0, 100])])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(4, 2, 128, "bf16"), (4, 1, 128, "fp16"), (3, 3, 72, "fp16"), (8, 1, 64, "bf16"),
                                            (2, 2, 96, "bf16"), (3, 1, 32, "fp16"), (2, 1, 32, "bf16"), (2, 2, 80, "fp16"),
                                            (2, 1, 64, "fp16")])
@pytest.mark.parametrize("causal", [True, False])
def test_packed(kq, lengths, past, Hq, Hkv, D, dtype, causal):
    cq, ck = cumulative(lengths), cumulative(past or lengths)
    Q = heads((int(cq[-1]), Hq, D), dtype, 1, 1.5)
    K, V = (heads((int(ck[-1]), Hkv, D), dtype, 2 + i) for i in range(2))
    o, tau = _expect(Q, K, V, cq, ck, causal, dtype)
    check(kq.attention(Q, K, V, on_gpu(cq), on_gpu(ck), causal=causal, precise=True), o, tau, dtype)
    if D == 128:
        check_codes(*kq.attention(Q, K, V, on_gpu(cq), on_gpu(ck), causal=causal, precise=True, fp8=True), o, tau)


@pytest.mark.parametrize("n", [8, 30, 700, 1500])           # whole, and split over the keys
@pytest.mark.parametrize("D", [32, 64, 80, 96, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_values_that_nearly_cancel(kq, n, D, dtype):
    K, V = (t.cuda() for t in pairs.rows(n, 2, D, dtype, dtype, n))
    Q = heads((7, 4, D), dtype, 4)
    for causal in (False, True):
        o, tau = _expect(Q, K, V, [0, 7], [0, n], causal, dtype)
        check(kq.attention(Q, K, V, causal=causal, precise=True), o, tau, dtype)
    if n == 8:                                              # and the other form is another
        assert not np.array_equal(raw(kq.attention(Q, K, V, precise=True)), raw(kq.attention(Q, K, V)))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_every_number_of_a_weight(kq, dtype):
    q, k, v = pairs.triples(64, dtype, 3)
    cq, ck = on_gpu(cumulative([1] * 64)), on_gpu(cumulative([3] * 64))
    O = kq.attention(q[:, None].cuda().contiguous(), k.reshape(192, 1, 32).cuda(), v.reshape(192, 1, 32).cuda(), cq, ck, scale=1.0,
                     precise=True)
    for b in range(64):
        o, tau = pairs.expect_triple(*(t[b].double().numpy() for t in (q, k, v)))
        check(O[b, 0], o, tau, dtype, f"sequence {b}")


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64)])
def test_not_finite(kq, dtype, D):
    """Infinities and NaN that are seen, and that are not."""
    cq = cumulative([100, 150, 30])
    Q, K, V = heads((280, 2, D), dtype, 20), heads((280, 1, D), dtype, 21), heads((280, 1, D), dtype, 22)
    V[160, 0, 3], V[170, 0, 4], V[180, 0, 4], V[190, 0, 5] = float("nan"), float("inf"), float("-inf"), float("inf")
    K[200, 0, 7] = float("nan")
    o, tau = _expect(Q, K, V, cq, cq, True, dtype)
    assert np.isposinf(o[175, 0, 4]) and np.isfinite(o[:160]).all() and np.isfinite(o[250:]).all()
    check(kq.attention(Q, K, V, on_gpu(cq), precise=True), o, tau, dtype)


def test_small_weights(kq):
    """One key far above 3000 others, whose values alone count: fp16 weights of 2^-23 of the largest."""
    n = 3000
    Q, K, V = torch.zeros(1, 1, 64), torch.zeros(n, 1, 64), 1.0 + 0.5 * torch.rand(n, 1, 64, generator=torch.Generator().manual_seed(0))
    Q[0, 0, 0], K[:, 0, 0], K[1234, 0, 0], V[1234] = 1.0, torch.linspace(-0.5, 0.5, n), 16.0, 0.0
    for T in (1, 300):                                      # split, and not
        q, k, v = Q.half().cuda().expand(T, 1, 64).contiguous(), K.half().cuda(), V.half().cuda()
        o, tau = _expect(q[:2], k, v, [0, len(q[:2])], [0, n], False, "fp16", 1.0)
        check(kq.attention(q, k, v, causal=False, scale=1.0, precise=True)[:2], o, tau, "fp16")


def test_captured_and_given_stream(kq):
    """A precise call replayed from a graph, and one on a given stream, give the eager call's bits."""
    cu = on_gpu(cumulative([100, 60, 40]))
    Q, K, V = heads((200, 4, 128), "bf16", 50), heads((200, 2, 128), "bf16", 51), heads((200, 2, 128), "bf16", 52)
    kq.attention(Q, K, V, cu, precise=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O = kq.attention(Q, K, V, cu, precise=True)
    for n in range(3):
        Q.copy_(heads((200, 4, 128), "bf16", 53 + n))
        graph.replay()
        ref = kq.attention(Q, K, V, cu, precise=True)
        torch.cuda.synchronize()
        side = kq.attention(Q, K, V, cu, precise=True, stream=torch.cuda.Stream())
        torch.cuda.synchronize()
        assert np.array_equal(raw(O), raw(ref)) and np.array_equal(raw(side), raw(ref))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,Tk", [(150, 150), (6, 2000)])
def test_default(kq, dtype, T, Tk):
    """Codes are precise unless the caller says otherwise, 16-bit outputs only if it does."""
    Q, (K, V) = heads((T, 4, 128), dtype, 60), (t.cuda() for t in pairs.rows(Tk, 2, 128, dtype, dtype, 61))
    o, tau = _expect(Q, K, V, [0, T], [0, Tk], True, dtype)
    codes, scales = kq.attention(Q, K, V, fp8=True)
    check_codes(codes, scales, o, tau)
    for a, b in zip((codes, scales), kq.attention(Q, K, V, fp8=True, precise=True)):
        assert np.array_equal(raw(a), raw(b))
    assert not np.array_equal(raw(codes), raw(kq.attention(Q, K, V, fp8=True, precise=False)[0]))
    assert np.array_equal(raw(kq.attention(Q, K, V)), raw(kq.attention(Q, K, V, precise=False)))
    assert not np.array_equal(raw(kq.attention(Q, K, V)), raw(kq.attention(Q, K, V, precise=True)))
