"""GPU parity of the paged attention at the precision of its weights, several 16-bit numbers each: on values that nearly cancel
(tolerances, and what they tell apart: tests/paged_pairs.py, tests/test_paged_precision_host.py), and in general."""

import numpy as np
import pytest

from oracle import attention as oracle
from tests import paged_pairs as pairs
from tests.attn_util import Cache, check, check_codes, cumulative, dbl, heads, on_gpu, raw, widened

pytestmark = pytest.mark.gpu


def _filled(kq, lengths, Hkv, D, dtype, cache, width, seed, new=None):
    """A cache whose sequences hold pairs that nearly cancel, or `new`."""
    c = Cache(lengths, Hkv, D, 16, dtype, cache, seed, width=width)
    new = new or [pairs.rows(n, Hkv, D, dtype, cache, seed + i) for i, n in enumerate(lengths)]
    K, V = (on_gpu(np.concatenate([t[i].float().numpy() for t in new])).to(new[0][0].dtype) for i in (0, 1))
    kq.cache_append(K, V, *c.args(), cu=on_gpu(cumulative(lengths)), **c.scales())
    if cache == "fp8":
        c.k64, c.v64 = (widened(raw(a).reshape(a.shape), raw(s).reshape(s.shape)) for a, s in ((c.k, c.ks), (c.v, c.vs)))
    else:
        c.k64, c.v64 = dbl(c.k), dbl(c.v)
    return c


def _expect(Q, c, dtype, cache):
    return oracle.paged(dbl(Q), c.k64, c.v64, c.table, c.lengths, float(np.float32(Q.shape[2] ** -0.5)), *pairs.WEIGHT[dtype, cache])


# whole heads by four wavefronts and by two, and dealt to runs that are joined 16 rows at a time and by four heads
@pytest.mark.parametrize("lengths,Hkv,width", [([8, 30, 17, 130, 600], 2, None), ([8, 17, 30, 55] * 75, 8, None),
                                               ([700, 900], 1, 300), ([8, 17, 30, 300] * 10 + [900], 2, 80)])
@pytest.mark.parametrize("dtype,cache", pairs.KINDS)
@pytest.mark.parametrize("D,group", [(128, 4), (64, 2)])
def test_values_that_nearly_cancel(kq, lengths, Hkv, width, dtype, cache, D, group):
    c = _filled(kq, lengths, Hkv, D, dtype, cache, width, 100)
    Q = heads((len(lengths), group * Hkv, D), dtype, 3)
    some = slice(None) if len(lengths) < 60 else slice(0, 40)               # the oracle takes its time
    o, tau = oracle.paged(dbl(Q)[some], c.k64, c.v64, c.table[some], c.lengths[some], float(np.float32(D ** -0.5)),
                          *pairs.WEIGHT[dtype, cache])
    check(kq.paged_attention(Q, *c.args(), **c.scales())[some], o, tau, dtype)
    if D == 128:
        codes, scales = kq.paged_attention(Q, *c.args(), **c.scales(), fp8=True)
        check_codes(codes[some], scales[some], o, tau)


@pytest.mark.parametrize("Hq,Hkv,D,page", [(4, 1, 128, 16), (20, 1, 64, 48), (6, 2, 96, 32), (5, 5, 112, 16), (33, 1, 128, 16)])
@pytest.mark.parametrize("dtype,cache", pairs.KINDS)
@pytest.mark.parametrize("width", [None, 200])
def test_one_token(kq, Hq, Hkv, D, page, dtype, cache, width):
    lengths = [1, 0, 15, 16, 17, 127, 128, 129, 300, 33, 0, 700]
    c = Cache(lengths, Hkv, D, page, dtype, cache, 1, width=width)
    Q = heads((len(lengths), Hq, D), dtype, 2, 1.5)
    o, tau = _expect(Q, c, dtype, cache)
    check(kq.paged_attention(Q, *c.args(), **c.scales()), o, tau, dtype)
    if D == 128:
        check_codes(*kq.paged_attention(Q, *c.args(), **c.scales(), fp8=True), o, tau)


@pytest.mark.parametrize("dtype,cache", pairs.KINDS)
@pytest.mark.parametrize("width", [None, 100])
def test_every_number_of_a_weight(kq, dtype, cache, width):
    q, k, v = pairs.triples(64, dtype, 3)
    c = _filled(kq, [3] * 64, 1, 32, dtype, cache, width, 5, [(k[b][:, None], v[b][:, None]) for b in range(64)])
    O = kq.paged_attention(q[:, None].cuda().contiguous(), *c.args(), **c.scales(), scale=1.0)
    for b in range(64):
        o, tau = pairs.expect_triple(q[b].double().numpy(), *(pairs.cached(t[b], cache) for t in (k, v)))
        check(O[b, 0], o, tau, dtype, f"sequence {b}")
