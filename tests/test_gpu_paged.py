"""GPU parity of the paged cache, its filling and the attention of one new token, against the float64 oracle."""

import numpy as np
import pytest
import torch

from oracle import attention as oracle
from tests.attn_util import DT, WEIGHT, Cache, check, check_codes, cumulative, dbl, heads, on_gpu, quantized, raw

pytestmark = pytest.mark.gpu

LENGTHS = [1, 0, 15, 16, 17, 127, 128, 129, 300, 33, 0, 700]


def _expect(Q, c, dtype, cache, scale=None):
    scale = Q.shape[2] ** -0.5 if scale is None else scale
    return oracle.paged(dbl(Q), c.k64, c.v64, c.table, c.lengths, np.float32(scale).astype(float), *WEIGHT[dtype, cache])


@pytest.mark.parametrize("Hq,Hkv,D,page,dtype,cache", [
    (4, 1, 128, 16, "bf16", "bf16"), (8, 2, 128, 32, "fp16", "fp16"), (2, 2, 64, 16, "bf16", "bf16"),
    (16, 1, 128, 64, "bf16", "fp8"), (6, 2, 128, 16, "fp16", "fp8"), (20, 1, 64, 48, "fp16", "fp8"), (3, 1, 72, 16, "fp16", "fp16"),
    (33, 1, 128, 16, "bf16", "bf16"), (2, 1, 32, 16, "bf16", "fp8"), (4, 4, 96, 128, "fp16", "fp8"), (2, 1, 8, 16, "fp16", "fp16"),
    (5, 5, 112, 16, "bf16", "fp8"), (40, 2, 64, 16, "bf16", "bf16")])
def test_one_token(kq, Hq, Hkv, D, page, dtype, cache):
    c = Cache(LENGTHS, Hkv, D, page, dtype, cache, 1)
    Q = heads((len(LENGTHS), Hq, D), dtype, 2, 1.5)
    O = kq.paged_attention(Q, *c.args(), **c.scales())
    check(O, *_expect(Q, c, dtype, cache), dtype)


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp8"), ("fp16", "fp8")])
@pytest.mark.parametrize("lengths", [[5000], [1], [0], [700, 3000, 0, 129, 2047]])
def test_split(kq, lengths, dtype, cache):
    """Few sequences, so that runs share heads; codes too."""
    c = Cache(lengths, 2, 128, 16, dtype, cache, 3)
    Q = heads((len(lengths), 6, 128), dtype, 4, 1.5)
    o, tau = _expect(Q, c, dtype, cache)
    check(kq.paged_attention(Q, *c.args(), **c.scales()), o, tau, dtype)
    check_codes(*kq.paged_attention(Q, *c.args(), **c.scales(), fp8=True), o, tau)


@pytest.mark.parametrize("width", [None, 70, 200])          # whole heads, by the table's width; else dealt to runs
@pytest.mark.parametrize("Hkv,D,cache", [(1, 64, "fp16"), (4, 64, "fp16"), (2, 128, "fp16"), (8, 64, "fp8")])
def test_many_sequences(kq, Hkv, D, cache, width):
    """More sequences than a wavefront has lanes and than there are compute units, most of them short, some empty
    (the first and last among them)."""
    rng = np.random.default_rng(5)
    lengths = [int(n) for n in rng.integers(0, 60, size=300)]
    lengths[0] = lengths[64] = lengths[299] = 0
    lengths[77], lengths[200] = 900, 400
    c = Cache(lengths, Hkv, D, 16, "fp16", cache, 6, width=width)
    Q = heads((300, 2 * Hkv, D), "fp16", 7)
    check(kq.paged_attention(Q, *c.args(), **c.scales()), *_expect(Q, c, "fp16", cache), "fp16")


def test_no_keys_at_all(kq):
    for width in (4, 300):
        c = Cache([0, 0, 0], 2, 64, 16, "bf16", "bf16", 6, width=width)
        O = torch.full((3, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        kq.paged_attention(heads((3, 4, 64), "bf16", 7), *c.args(), O=O)
        assert (O == 0).all()


@pytest.mark.parametrize("cache", ["fp16", "fp8"])
def test_pages_that_are_not_there(kq, cache):
    """Entries outside the cache hide their tokens; lengths outside the table are held to it."""
    c = Cache([200, 90, 40], 2, 64, 16, "fp16", cache, 8, hole=True)
    c.lengths = np.array([100000, -3, 40], np.int32)
    c.table[0, 13:] = -1
    o_len = np.minimum(np.maximum(c.lengths, 0), c.width * 16)
    Q = heads((3, 4, 64), "fp16", 9)
    # the last page of sequence 0 ends with rows that hold no token
    for t in ((c.k, c.v) if cache == "fp16" else ()):
        t[torch.isnan(t)] = 0.5
    if cache == "fp16":
        c.k64, c.v64 = dbl(c.k), dbl(c.v)
    else:
        for s, codes in ((c.ks, c.k), (c.vs, c.v)):
            codes.view(torch.uint8)[(s == 255)[..., None].expand(codes.shape)] = 0x38
            s[s == 255] = 127
        from tests.attn_util import widened
        c.k64, c.v64 = widened(raw(c.k).reshape(c.k.shape), raw(c.ks).reshape(c.ks.shape)), widened(raw(c.v).reshape(c.v.shape), raw(c.vs).reshape(c.vs.shape))
    o, tau = _expect(Q, c, "fp16", cache)
    assert (o_len == [c.width * 16, 0, 40]).all() and (o[1] == 0).all()
    check(kq.paged_attention(Q, *c.args(), **c.scales()), o, tau, "fp16")


def test_shared_pages_and_wide_tables(kq):
    """Sequences that share their first pages; a table wider than any sequence, with entries that are never read."""
    c = Cache([100, 100], 2, 128, 16, "bf16", "bf16", 10, width=40)
    c.table[1, :4] = c.table[0, :4]
    c.table[:, 20:] = 1 << 30
    Q = heads((2, 4, 128), "bf16", 11)
    check(kq.paged_attention(Q, *c.args()), *_expect(Q, c, "bf16", "bf16"), "bf16")


def test_nan_that_is_seen(kq):
    c = Cache([50, 40], 1, 64, 16, "bf16", "bf16", 12)
    c.v[c.table[0, 1], 0, 3, 5] = float("nan")
    c.k[c.table[1, 0], 0, 0, 0] = float("nan")
    c.k64, c.v64 = dbl(c.k), dbl(c.v)
    Q = heads((2, 2, 64), "bf16", 13)
    o, tau = _expect(Q, c, "bf16", "bf16")
    assert np.isnan(o[0, 0, 5]) and np.isfinite(o[0, 0, 4]) and np.isnan(o[1]).all()
    check(kq.paged_attention(Q, *c.args()), o, tau, "bf16")


@pytest.mark.parametrize("dtype,cache", [("fp16", "fp16"), ("bf16", "bf16"), ("fp16", "fp8")])
def test_many_small_weights(kq, dtype, cache):
    """One key far above 30000 others, whose values alone count: weights near 2^-23 of the largest keep their
    precision."""
    n = 30000
    c = Cache([n], 1, 64, 16, dtype, cache, 80)
    q = torch.zeros((1, 1, 64), dtype=DT[dtype], device="cuda")
    q[0, 0, 0] = 1.0
    k = torch.zeros((n, 64), device="cuda")
    k[:, 0] = torch.linspace(-0.5, 0.5, n, device="cuda")
    k[4321, 0] = 16.0
    v = 1.0 + 0.5 * torch.rand((n, 64), device="cuda")
    v[4321] = 0.0
    c.lengths[:] = n
    kq.cache_append(k.to(DT[dtype])[:, None], v.to(DT[dtype])[:, None], *c.args(), cu=on_gpu(np.array([0, n], np.int32)), **c.scales())
    if cache == "fp8":
        from tests.attn_util import widened
        c.k64, c.v64 = (widened(raw(a).reshape(a.shape), raw(s).reshape(s.shape)) for a, s in ((c.k, c.ks), (c.v, c.vs)))
    else:
        c.k64, c.v64 = dbl(c.k), dbl(c.v)
    o, tau = _expect(q, c, dtype, cache, 1.0)
    assert 0.001 < o.min() < o.max() < 0.02
    check(kq.paged_attention(q, *c.args(), **c.scales(), scale=1.0), o, tau, dtype)
    if cache != "fp8":
        K, V = (torch.from_numpy(t).to(DT[dtype]).cuda() for t in (c.k64, c.v64))
        rows = [t[torch.from_numpy(c.table[0]).long().cuda()].transpose(1, 2).reshape(-1, 1, 64)[:n].contiguous() for t in (K, V)]
        check(kq.attention(q, *rows, scale=1.0), o, tau, dtype)


def test_scale_byte_that_is_nan(kq):
    """Byte 255 makes NaN what uses it, whatever the codes."""
    c = Cache([40, 40, 40], 1, 64, 16, "bf16", "fp8", 81)
    c.ks[c.table[0, 1], 0, 3] = 255
    c.vs[c.table[1, 2], 0, 1] = 255
    y = dbl(kq.paged_attention(heads((3, 2, 64), "bf16", 82), *c.args(), **c.scales()))
    assert np.isnan(y[:2]).all() and np.isfinite(y[2]).all()


def test_queries_views(kq):
    c = Cache([70, 30, 200], 2, 128, 16, "bf16", "bf16", 14)
    qkv = heads((3, 8, 128), "bf16", 15)
    Q = qkv[:, :4]
    ref = kq.paged_attention(Q.contiguous(), *c.args())
    assert np.array_equal(raw(kq.paged_attention(Q, *c.args())), raw(ref))
    turned = Q.transpose(0, 1).contiguous().transpose(0, 1)
    assert np.array_equal(raw(kq.paged_attention(turned, *c.args())), raw(ref))


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_cache_past_32_bits(kq, cache):
    """Pages whose offsets pass 2^32 bytes (and, in the 8-bit cache, 2^31 rows of scales do not exist below them)."""
    page, D = 64, 128
    pages = (9 << 30) // (page * D * (1 if cache == "fp8" else 2))
    small = Cache([150, 90], 1, D, page, "bf16", cache, 16)
    big = {}
    for name, t in (("k", small.k), ("v", small.v)):
        big[name] = torch.zeros((pages, 1, page, D), dtype=t.dtype, device="cuda")
        big[name].view(torch.uint8)[pages - small.pages:] = t.view(torch.uint8)
    scales = {}
    if cache == "fp8":
        for name, t in small.scales().items():
            scales[name] = torch.full((pages, 1, page), 127, dtype=torch.uint8, device="cuda")
            scales[name][pages - small.pages:] = t
    table = small.table + np.where(small.table >= 0, pages - small.pages, 0).astype(np.int32)
    Q = heads((2, 4, D), "bf16", 17)
    O = kq.paged_attention(Q, big["k"], big["v"], on_gpu(table), on_gpu(small.lengths), **scales)
    check(O, *_expect(Q, small, "bf16", cache), "bf16")
    new = heads((2, 1, D), "bf16", 18)
    kq.cache_append(new, new, big["k"], big["v"], on_gpu(table), on_gpu(small.lengths), **scales)
    kq.cache_append(new, new, *small.args(), **small.scales())
    assert np.array_equal(raw(big["k"][pages - small.pages:]), raw(small.k)) and np.array_equal(raw(big["v"][pages - small.pages:]), raw(small.v))


# ---- filling

def _append_expect(c, K, V, cu, cache, dtype):
    if cache != "fp8":
        bits = [t.view(torch.int16).cpu().numpy() for t in (c.k, c.v, K, V)]
        put = lambda to, new: to.__setitem__(slice(None), new)
        return [oracle.append(n, o, c.table, c.lengths, cu, put) for o, n in zip(bits[:2], bits[2:])]
    out = []
    for codes, scales, new in ((c.k, c.ks, K), (c.v, c.vs, V)):
        q, s = quantized(dbl(new))
        put = lambda to, new: to.__setitem__(slice(None), new)
        out.append(oracle.append(q, raw(codes).reshape(codes.shape), c.table, c.lengths, cu, put))
        out.append(oracle.append(s, raw(scales).reshape(scales.shape), c.table, c.lengths, cu, put))
    return out


@pytest.mark.parametrize("Hkv,D,page,dtype,cache", [
    (2, 128, 16, "bf16", "bf16"), (1, 72, 32, "fp16", "fp16"), (3, 64, 16, "bf16", "fp8"), (8, 128, 64, "fp16", "fp8"),
    (5, 8, 16, "bf16", "bf16"), (2, 16, 16, "fp16", "fp8"), (1, 112, 48, "bf16", "fp8")])
@pytest.mark.parametrize("form", ["packed", "tokens"])
def test_append(kq, Hkv, D, page, dtype, cache, form):
    """Every byte of the cache: the new rows, and all others as they were."""
    lengths = [20, 3, 64, 1, 130, 90]
    new = [1] * 6 if form == "tokens" else [20, 0, 7, 1, 100, 2]
    c = Cache(lengths, Hkv, D, page, dtype, cache, 20, spare=3)
    T = sum(new)
    kv = heads((T, 2 * Hkv, D), dtype, 21)
    kv[T // 2] *= 50
    kv[0, 0] = 0
    K, V = kv[:, :Hkv], kv[:, Hkv:]
    if cache == "fp8":
        V[T - 1, 0, 3] = float("nan")
    cu = cumulative(new)
    expect = _append_expect(c, K.contiguous(), V.contiguous(), cu, cache, dtype)
    out = kq.cache_append(K, V, *c.args(), **c.scales(), **({} if form == "tokens" else dict(cu=on_gpu(cu))))
    assert out[0] is c.k and out[1] is c.v
    got = [c.k, c.v] if cache != "fp8" else [c.k, c.ks, c.v, c.vs]
    for g, e in zip(got, expect):
        assert np.array_equal(raw(g).reshape(-1), np.ascontiguousarray(e).view(np.uint8).reshape(-1))


def test_append_drops_what_has_no_place(kq):
    """Positions below zero or beyond the table, pages that are not there, rows of no sequence."""
    c = Cache([40, 16, 33, 5], 2, 64, 16, "fp16", "fp16", 22)
    c.lengths = np.array([40, 2000, 33, 5], np.int32)
    c.table[2, 1], c.table[2, 2] = -1, c.pages
    cu = np.array([3, 10, 20, 60, 90], np.int32)              # sequence 3: 30 new tokens of 5
    K, V = heads((120, 2, 64), "fp16", 23), heads((120, 2, 64), "fp16", 24)
    expect = _append_expect(c, K, V, cu, "fp16", "fp16")
    kq.cache_append(K, V, *c.args(), cu=on_gpu(cu))
    for g, e in zip((c.k, c.v), expect):
        assert np.array_equal(raw(g).reshape(-1), np.ascontiguousarray(e).view(np.uint8).reshape(-1))


@pytest.mark.parametrize("B", [150, 4500])
def test_append_many_sequences(kq, B):
    rng = np.random.default_rng(25)
    new = [int(n) for n in rng.integers(0, 4, size=B)]
    c = Cache([n + 5 for n in new], 1, 64, 16, "bf16", "bf16", 26)
    K, V = heads((sum(new), 1, 64), "bf16", 27), heads((sum(new), 1, 64), "bf16", 28)
    expect = _append_expect(c, K, V, cumulative(new), "bf16", "bf16")
    kq.cache_append(K, V, *c.args(), cu=on_gpu(cumulative(new)))
    for g, e in zip((c.k, c.v), expect):
        assert np.array_equal(raw(g).reshape(-1), np.ascontiguousarray(e).view(np.uint8).reshape(-1))


# ---- together

@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_block(kq, cache):
    """Norm, projection, filling, attention and output projection of a batch of prompts, then of one more token each:
    the prompts' attention of the last tokens and the cache's agree."""
    Hq, Hkv, D, K = 4, 2, 128, 256
    g = torch.Generator(device="cuda").manual_seed(30)
    def weights(n, k):
        return kq.quantize_fp8((torch.randn(n, k, device="cuda", generator=g) * k ** -0.5).to(torch.bfloat16))
    wqkv, wout = weights((Hq + 2 * Hkv) * D, K), weights(K, Hq * D)
    gamma = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    prompts = [37, 1, 150]
    X = torch.randn(sum(prompts), K, device="cuda", generator=g).to(torch.bfloat16)
    c = Cache([n + 1 for n in prompts], Hkv, D, 16, "bf16", cache, 31)

    def qkv(x):
        codes, scales, _ = kq.rmsnorm_quantize_fp8(x, gamma)
        y = kq.fp8_linear(codes, scales, *wqkv, dtype=torch.bfloat16).view(len(x), Hq + 2 * Hkv, D)
        return y.split((Hq, Hkv, Hkv), dim=1)
    cu = cumulative(prompts)
    Q, Kn, Vn = qkv(X)
    table, lengths = on_gpu(c.table), on_gpu(np.array(prompts, np.int32))
    kq.cache_append(Kn, Vn, c.k, c.v, table, lengths, on_gpu(cu), **c.scales())
    out = kq.fp8_linear(*kq.attention(Q, Kn, Vn, on_gpu(cu), fp8=True), *wout, dtype=torch.bfloat16)
    assert out.shape == X.shape and torch.isfinite(out).all()
    # the last tokens of the prompts, from the cache
    last = torch.from_numpy(cu[1:].astype(np.int64) - 1).cuda()
    fresh = dbl(kq.attention(Q, Kn, Vn, on_gpu(cu)))[cu[1:] - 1]
    held = dbl(kq.paged_attention(Q[last], c.k, c.v, table, lengths, **c.scales()))
    # 8-bit keys and values: half a step of 2^-4 each; the scores of these queries stay below 4
    far = np.abs(fresh - held).max()
    assert far <= (0.02 if cache == "bf16" else 0.5), far
    # one more token
    x = torch.randn(3, K, device="cuda", generator=g).to(torch.bfloat16)
    q, k, v = qkv(x)
    lengths += 1
    kq.cache_append(k, v, c.k, c.v, table, lengths, **c.scales())
    if cache == "bf16":
        c.k64, c.v64 = dbl(c.k), dbl(c.v)
    else:
        from tests.attn_util import widened
        c.k64, c.v64 = (widened(raw(a).reshape(a.shape), raw(s).reshape(s.shape)) for a, s in ((c.k, c.ks), (c.v, c.vs)))
    c.lengths = lengths.cpu().numpy()
    o, tau = _expect(q, c, "bf16", cache)
    check(kq.paged_attention(q, c.k, c.v, table, lengths, **c.scales()), o, tau, "bf16")
    codes, scales = kq.paged_attention(q, c.k, c.v, table, lengths, **c.scales(), fp8=True)
    check_codes(codes, scales, o, tau)
    y = kq.fp8_linear(codes, scales, *wout, dtype=torch.bfloat16)
    assert y.shape == x.shape and torch.isfinite(y).all()


@pytest.mark.parametrize("width", [8, 100])                  # not split, and split
def test_captured_step(kq, width):
    """A step (append, attention) captured and replayed on new tokens and lengths, with eager work between."""
    lengths = [40, 7, 90]
    c = Cache([n + 8 for n in lengths], 2, 128, 16, "bf16", "bf16", 40, width=width)
    k2, v2 = c.k.clone(), c.v.clone()
    table, ln = on_gpu(c.table), on_gpu(np.array(lengths, np.int32))
    qkv = heads((3, 8, 128), "bf16", 41)
    Q, K, V = qkv.split((4, 2, 2), dim=1)
    nb = kq.paged_attention_workspace_bytes(3, 4, 2, 128, c.width, 16)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")

    def step():
        ln.add_(1)
        kq.cache_append(K, V, c.k, c.v, table, ln)
        return kq.paged_attention(Q, c.k, c.v, table, ln, fp8=True, workspace=ws)
    step()
    ln.sub_(1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        codes, scales = step()
    torch.cuda.synchronize()
    ln2 = on_gpu(np.array(lengths, np.int32))
    for n in range(4):
        qkv.copy_(heads((3, 8, 128), "bf16", 42 + n))
        graph.replay()
        ln2 += 1
        kq.cache_append(K, V, k2, v2, table, ln2)
        a, b = kq.paged_attention(Q, k2, v2, table, ln2, fp8=True)
        torch.cuda.synchronize()
        assert np.array_equal(raw(a), raw(codes)) and np.array_equal(raw(b), raw(scales))
        assert torch.equal(ln, ln2)


def test_captured_prompt(kq):
    cu = on_gpu(cumulative([100, 60, 40]))
    Q, K, V = heads((200, 4, 128), "bf16", 50), heads((200, 2, 128), "bf16", 51), heads((200, 2, 128), "bf16", 52)
    kq.attention(Q, K, V, cu)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O = kq.attention(Q, K, V, cu)
    for n in range(3):
        Q.copy_(heads((200, 4, 128), "bf16", 53 + n))
        cu.copy_(on_gpu(cumulative([40 + n, 120, 40 - n])))
        graph.replay()
        ref = kq.attention(Q, K, V, cu)
        torch.cuda.synchronize()
        assert np.array_equal(raw(O), raw(ref))


def test_two_streams(kq):
    """Calls on two streams at once, each with its own workspace."""
    c = Cache([3000, 50, 700], 2, 128, 16, "bf16", "bf16", 60)
    Q = [heads((3, 4, 128), "bf16", 61 + i) for i in range(2)]
    args = c.args()
    ref = [raw(kq.paged_attention(q, *args)) for q in Q]
    P = [heads((400, 4, 128), "bf16", 63 + i) for i in range(2)]
    pref = [raw(kq.attention(p, p[:, :2], p[:, 2:])) for p in P]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        out = [(kq.paged_attention(q, *args, stream=s), kq.attention(p, p[:, :2], p[:, 2:], stream=s))
               for q, p, s in zip(Q, P, streams)]
        torch.cuda.synchronize()
        for (a, b), r, pr in zip(out, ref, pref):
            assert np.array_equal(raw(a), r) and np.array_equal(raw(b), pr)


def test_memory_of_a_given_stream(kq):
    """Outputs and workspaces that calls make on a given stream are memory of that stream."""
    c = Cache([3000, 50], 2, 128, 16, "bf16", "bf16", 85)
    args, Q = c.args(), heads((2, 4, 128), "bf16", 86)
    K, V = heads((3000, 2, 128), "bf16", 87), heads((3000, 2, 128), "bf16", 88)
    calls = [lambda s: kq.paged_attention(Q, *args, stream=s), lambda s: kq.paged_attention(Q, *args, fp8=True, stream=s),
             lambda s: kq.attention(Q, K, V, stream=s), lambda s: kq.attention(K, K, V, fp8=True, stream=s)]
    side = torch.cuda.Stream()
    for call in calls:
        expect = call(None)
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        before = {s["address"] for s in torch.cuda.memory_snapshot()}
        out = call(side)
        assert all(s["stream"] == side.cuda_stream for s in torch.cuda.memory_snapshot() if s["address"] not in before)
        torch.cuda.synchronize()
        for a, b in zip(expect if isinstance(expect, tuple) else (expect,), out if isinstance(out, tuple) else (out,)):
            assert np.array_equal(raw(a), raw(b))
        del out
    with torch.cuda.stream(torch.cuda.Stream()):
        assert kq.cache_append(K[:2], V[:2], *args, stream=side)[0] is c.k
    torch.cuda.synchronize()


def test_refusals(kq):
    c = Cache([20, 30], 2, 128, 16, "bf16", "fp8", 70)
    Q = heads((2, 4, 128), "bf16", 71)
    k, v, table, ln = c.args()
    for bad, match in (((k, v, table, ln, dict(kscales=c.ks)), "go together"), ((k, v, table, ln, {}), "bfloat16"),
                       ((k, v, table.long(), ln, c.scales()), "int32"), ((k, v, table[:1], ln, c.scales()), "shape"),
                       ((k, v, table, ln[:1], c.scales()), "shape"), ((k[0], v, table, ln, c.scales()), "4-D"),
                       ((k, v[:1], table, ln, c.scales()), "shape"), ((k, v, table[0], ln, c.scales()), "2-D")):
        with pytest.raises(ValueError, match=match):
            kq.paged_attention(Q, *bad[:4], **bad[4])
        with pytest.raises(ValueError):
            kq.cache_append(Q[:, :2], Q[:, 2:], *bad[:4], **bad[4])
    long = table[:, :1].expand(2, 300).contiguous()
    with pytest.raises(kq.KQError):
        kq.paged_attention(Q, k, v, long, ln, **c.scales(), workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        kq.cache_append(Q[:, :2], Q[:, 2:], k, v, table, ln, on_gpu(np.zeros(2, np.int32)), **c.scales())
    with pytest.raises(kq.KQError):                            # three tokens of two sequences, and no cu
        kq.cache_append(heads((3, 2, 128), "bf16", 72), heads((3, 2, 128), "bf16", 73), k, v, table, ln, **c.scales())
