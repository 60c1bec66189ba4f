"""GPU parity of attention over packed sequences against the float64 oracle (tolerances: oracle/attention.py and
attn_util.WEIGHT)."""

import numpy as np
import pytest
import torch

from oracle import attention as oracle
from tests.attn_util import DT, WEIGHT, check, check_codes, cumulative, dbl, heads, on_gpu, raw

pytestmark = pytest.mark.gpu

# query lengths, key lengths (None: the same)
LENGTHS = {
    "one": ([1], None),
    "single": ([200], None),
    "tile": ([128, 64], None),
    "ragged": ([5, 0, 131, 1, 257, 64], None),
    "cross": ([70, 3, 129], [20, 300, 1]),
    "behind": ([40, 1, 130], [200, 77, 131]),        # keys that were there before
    "short": ([150, 9], [64, 3]),                     # causal: the first queries see nothing
    "keyless": ([17, 33, 2], [0, 65, 0]),
}


def _case(name, Hq, Hkv, D, dtype, seed=0, spread=1.5):
    q, k = LENGTHS[name]
    k = q if k is None else k
    return (heads((sum(q), Hq, D), dtype, seed, spread), heads((sum(k), Hkv, D), dtype, seed + 1),
            heads((sum(k), Hkv, D), dtype, seed + 2), cumulative(q), cumulative(k))


def _expect(Q, K, V, cq, ck, causal, dtype, scale=None):
    scale = Q.shape[2] ** -0.5 if scale is None else scale
    return oracle.attention(dbl(Q), dbl(K), dbl(V), cq, ck, causal, np.float32(scale).astype(np.float64), *WEIGHT[dtype, dtype])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name,Hq,Hkv,D,dtype", [
    ("one", 2, 1, 128, "bf16"), ("single", 4, 2, 128, "bf16"), ("single", 8, 8, 64, "fp16"), ("tile", 4, 1, 128, "fp16"),
    ("ragged", 3, 3, 72, "fp16"), ("ragged", 4, 2, 128, "bf16"), ("ragged", 8, 1, 64, "bf16"), ("cross", 2, 2, 72, "fp16"),
    ("cross", 16, 2, 32, "bf16"), ("behind", 4, 2, 128, "bf16"), ("behind", 2, 1, 96, "fp16"), ("short", 2, 1, 128, "fp16"),
    ("short", 2, 2, 40, "bf16"), ("keyless", 2, 1, 128, "bf16"), ("keyless", 3, 1, 8, "fp16"), ("ragged", 2, 1, 80, "bf16"),
    ("ragged", 2, 2, 112, "fp16"), ("single", 1, 1, 24, "bf16"), ("ragged", 8, 2, 48, "fp16")])
def test_packed(kq, name, Hq, Hkv, D, dtype, causal):
    Q, K, V, cq, ck = _case(name, Hq, Hkv, D, dtype)
    if len(K) == 0:
        return
    O = kq.attention(Q, K, V, on_gpu(cq), on_gpu(ck), causal=causal)
    check(O, *_expect(Q, K, V, cq, ck, causal, dtype), dtype)


def test_no_cu_is_one_sequence(kq):
    Q, K, V, cq, ck = _case("single", 4, 2, 64, "bf16")
    for causal in (True, False):
        a = kq.attention(Q, K, V, causal=causal, scale=0.2)
        b = kq.attention(Q, K, V, on_gpu(cq), causal=causal, scale=0.2)
        assert np.array_equal(raw(a), raw(b))
        check(a, *_expect(Q, K, V, cq, ck, causal, "bf16", 0.2), "bf16")


@pytest.mark.parametrize("Hq,Hkv,name", [(4, 2, "ragged"), (5, 1, "short"), (8, 8, "behind"), (3, 3, "keyless"), (1, 1, "one")])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_codes(kq, Hq, Hkv, name, dtype):
    Q, K, V, cq, ck = _case(name, Hq, Hkv, 128, dtype, 5)
    codes, scales = kq.attention(Q, K, V, on_gpu(cq), on_gpu(ck), fp8=True)
    assert codes.shape == (len(Q), Hq * 128) and scales.shape == (len(Q), kq.fp8_scale_cols(Hq * 128))
    check_codes(codes, scales, *_expect(Q, K, V, cq, ck, True, dtype))


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 72)])
def test_many_tiles(kq, dtype, D):
    """A thousand keys and more: maxima that move in every tile, and the heads dealt over the dies (8 heads)."""
    Q, K, V = heads((1111, 8, D), dtype, 3, 2.0), heads((1111, 2, D), dtype, 4), heads((1111, 2, D), dtype, 5)
    ramp = torch.linspace(0.2, 4.0, 1111).to(DT[dtype]).cuda()[:, None, None]
    K = K * ramp
    O = kq.attention(Q, K, V)
    rows = np.r_[0:40, 500:530, 1060:1111]
    q, k, v = dbl(Q), dbl(K), dbl(V)
    for h in (0, 5, 7):
        o, tau = oracle.attend(q[rows, h], k[:, h // 4], v[:, h // 4], np.float32(D ** -0.5).astype(float), rows + 1, *WEIGHT[dtype, dtype])
        check(O[rows, h], o, tau, dtype, f"head {h}")


@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(4, 2, 128, "bf16"), (3, 3, 72, "fp16"), (8, 1, 64, "bf16"), (2, 1, 32, "fp16"),
                                            (2, 2, 96, "bf16")])
@pytest.mark.parametrize("causal", [True, False])
def test_split_keys(kq, Hq, Hkv, D, dtype, causal):
    """Few queries of many keys: split over the keys.  Sequences without keys, without queries, with fewer keys than
    queries, and rows of no sequence, among them."""
    q, k = [3, 0, 20, 1, 70, 5, 9], [1500, 40, 700, 0, 100, 130, 4]
    cq, ck = cumulative(q) + 2, cumulative(k) + 7
    T, Tk = int(cq[-1]) + 4, int(ck[-1]) + 9
    Q, K, V = heads((T, Hq, D), dtype, 70, 1.5), heads((Tk, Hkv, D), dtype, 71), heads((Tk, Hkv, D), dtype, 72)
    for t, c in ((Q, cq), (K, ck), (V, ck)):
        t[:c[0]] = float("nan")
        t[c[-1]:] = float("nan")
    K[ck[0]:ck[1]] *= torch.linspace(0.3, 3.0, 1500).to(DT[dtype]).cuda()[:, None, None]
    assert kq.attention_workspace_bytes(len(q), T, Tk, True, Hq, Hkv, D) > 0
    O = torch.full((T, Hq, D), 7.0, dtype=DT[dtype], device="cuda")
    kq.attention(Q, K, V, on_gpu(cq), on_gpu(ck), causal=causal, O=O)
    o, tau = _expect(Q, K, V, cq, ck, causal, dtype)
    o[:2] = o[-4:] = 7.0
    check(O, o, tau, dtype)
    if D == 128:
        codes, scales = kq.attention(Q, K, V, on_gpu(cq), on_gpu(ck), causal=causal, fp8=True)
        check_codes(codes[2:-4], scales[2:-4], o[2:-4], tau[2:-4])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_split_keys_hidden_nan(kq, dtype):
    """As test_hidden_nan_and_infinities, with the keys split; one sequence, no cu."""
    Q, K, V = heads((6, 2, 64), dtype, 80), heads((2000, 1, 64), dtype, 81), heads((2000, 1, 64), dtype, 82)
    V[1996, 0, 3], V[1997, 0, 4], V[100, 0, 9] = float("nan"), float("inf"), float("-inf")
    K[1998, 0, 7] = float("nan")
    assert kq.attention_workspace_bytes(1, 6, 2000, False, 2, 1, 64) > 0
    o, tau = _expect(Q, K, V, [0, 6], [0, 2000], True, dtype)
    assert np.isfinite(o[0, 0, 3]) and np.isnan(o[2, 0, 3]) and np.isneginf(o[0, 0, 9]) and np.isnan(o[4]).all()
    check(kq.attention(Q, K, V), o, tau, dtype)


def test_split_keys_workspace(kq):
    """A given workspace serves; one that is too small is refused."""
    Q, K, V = heads((5, 4, 128), "bf16", 90), heads((3000, 2, 128), "bf16", 91), heads((3000, 2, 128), "bf16", 92)
    ref = kq.attention(Q, K, V)
    nb = kq.attention_workspace_bytes(1, 5, 3000, False, 4, 2, 128)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    assert np.array_equal(raw(kq.attention(Q, K, V, workspace=ws)), raw(ref))
    with pytest.raises(kq.KQError):
        kq.attention(Q, K, V, workspace=ws[:nb - 256])
    with pytest.raises(ValueError):
        kq.attention(Q, K, V, workspace=ws.int())


def test_large_scores(kq):
    """Scores of tens of thousands: the softmax is one key's, whatever the order of the maxima."""
    Q, K, V, cq, ck = _case("single", 2, 2, 64, "fp16", 9)
    Q, K = Q * 60, K * 60
    O = kq.attention(Q, K, V, causal=False)
    check(O, *_expect(Q, K, V, cq, ck, False, "fp16"), "fp16")


def test_views(kq):
    """Strided views, a transposed layout and heads that repeat by a zero stride give the bits of copies."""
    T, Hq, Hkv, D = 190, 4, 2, 128
    qkv = heads((T, Hq + 2 * Hkv, D), "bf16", 11)
    Q, K, V = qkv.split((Hq, Hkv, Hkv), dim=1)
    ref = kq.attention(Q.contiguous(), K.contiguous(), V.contiguous())
    assert np.array_equal(raw(kq.attention(Q, K, V)), raw(ref))
    turned = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (Q, K, V)]
    assert not turned[0].is_contiguous()
    assert np.array_equal(raw(kq.attention(*turned)), raw(ref))
    one = kq.attention(Q, K[:, :1].expand(T, 4, D), V[:, :1].expand(T, 4, D))
    assert np.array_equal(raw(one), raw(kq.attention(Q, K[:, :1].contiguous(), V[:, :1].contiguous())))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
def test_hidden_nan_and_infinities(kq, dtype, D):
    """NaN and infinities at keys and values reach the queries that see them and no others; the neighbouring
    sequence's are not seen at all."""
    cq = cumulative([100, 150, 30])
    Q, K, V = heads((280, 2, D), dtype, 20), heads((280, 1, D), dtype, 21), heads((280, 1, D), dtype, 22)
    V[160, 0, 3], V[170, 0, 4], V[180, 0, 4], V[190, 0, 5] = float("nan"), float("inf"), float("-inf"), float("inf")
    K[200, 0, 7] = float("nan")
    o, tau = _expect(Q, K, V, cq, cq, True, dtype)
    assert np.isnan(o[170, 0, 3]) and np.isposinf(o[175, 0, 4]) and np.isnan(o[185, 0, 4]) and np.isnan(o[201]).all()
    assert np.isfinite(o[:160]).all() and np.isfinite(o[250:]).all()
    check(kq.attention(Q, K, V, on_gpu(cq)), o, tau, dtype)
    if D == 128:
        codes, scales = kq.attention(Q, K, V, on_gpu(cq), fp8=True)
        check_codes(codes, scales, o, tau)


def test_rows_outside_stay(kq):
    """Rows before, and behind, the sequences: neither read nor written."""
    Q, K, V = heads((300, 2, 128), "fp16", 30), heads((300, 2, 128), "fp16", 31), heads((300, 2, 128), "fp16", 32)
    for t in (Q, K, V):
        t[:10] = float("nan")
        t[210:] = float("nan")
    cu = np.array([10, 50, 50, 210], np.int32)
    O = torch.full((300, 2, 128), 7.0, dtype=torch.float16, device="cuda")
    assert kq.attention(Q, K, V, on_gpu(cu), O=O) is O
    o, tau = _expect(Q, K, V, cu, cu, True, "fp16")
    o[:10] = o[210:] = 7.0
    check(O, o, tau, "fp16")
    codes, scales = torch.full((300, 256), 3, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn), torch.full((300, 4), 9, dtype=torch.uint8, device="cuda")
    kq.attention(Q, K, V, on_gpu(cu), fp8=True, codes=codes, scales=scales)
    check_codes(codes[10:210], scales[10:210], o[10:210], tau[10:210])
    for s in (slice(0, 10), slice(210, 300)):
        assert (raw(codes[s]) == 3).all() and (raw(scales[s]) == 9).all()


@pytest.mark.parametrize("cq,ck", [([0, 500, 300], [0, 90, 40]), ([-5, 120, 60, 1 << 30], [7, 1 << 30, -9, 300]),
                                   ([200, 100, 0], [200, 100, 0]), ([300, 300], [0, 300])])
def test_entries_that_make_no_sense(kq, cq, ck):
    """Entries of cu out of range or order lead nowhere outside the tensors."""
    Q, K, V = heads((300, 2, 64), "bf16", 40), heads((300, 1, 64), "bf16", 41), heads((300, 1, 64), "bf16", 42)
    room = torch.full((900, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    kq.attention(Q, K, V, on_gpu(np.array(cq, np.int32)), on_gpu(np.array(ck, np.int32)), O=room[300:600])
    torch.cuda.synchronize()
    assert (room[:300] == 5).all() and (room[600:] == 5).all() and torch.isfinite(room).all()


@pytest.mark.parametrize("B,most", [(201, 9), (5000, 3)])
def test_many_sequences(kq, B, most):
    """More sequences than a wavefront has lanes, and than its square, some empty."""
    rng = np.random.default_rng(50)
    cu = cumulative(rng.integers(0, most, size=B))
    T = int(cu[-1])
    Q, K, V = heads((T, 2, 64), "fp16", 51), heads((T, 1, 64), "fp16", 52), heads((T, 1, 64), "fp16", 53)
    check(kq.attention(Q, K, V, on_gpu(cu)), *_expect(Q, K, V, cu, cu, True, "fp16"), "fp16")


def test_keys_past_32_bits(kq):
    """Tokens whose offsets pass 2^32 bytes."""
    T, D = 4200, 64
    big = torch.zeros((T, 1 << 20), dtype=torch.bfloat16, device="cuda")            # 2 MiB a token
    K, V = big[:, :D].unsqueeze(1), big[:, -D:].unsqueeze(1)
    K.copy_(heads((T, 1, D), "bf16", 60))
    V.copy_(heads((T, 1, D), "bf16", 61))
    Q = heads((2, 1, D), "bf16", 62)
    o, tau = _expect(Q, K, V, [0, 2], [0, T], True, "bf16")
    check(kq.attention(Q, K, V, on_gpu(np.array([0, 2], np.int32)), on_gpu(np.array([0, T], np.int32))), o, tau, "bf16")


def test_refusals(kq):
    Q, K = heads((4, 2, 64), "bf16", 1), heads((5, 2, 64), "bf16", 2)
    cu = on_gpu(np.array([0, 4], np.int32))
    for bad, match in ((dict(cu_k=cu), "without cu_q"), (dict(cu_q=cu), "cu_k must be given"), (dict(cu_q=cu.long(), cu_k=cu), "int32"),
                       (dict(fp8=True), "heads of 128"), (dict(codes=Q), "without fp8"), (dict(O=Q[:3]), "shape"),
                       (dict(fp8=True, O=Q), "with fp8")):
        with pytest.raises(ValueError, match=match):
            kq.attention(Q, K, K, **bad)
    with pytest.raises(ValueError, match="shape"):
        kq.attention(Q, K, K[:4])
    with pytest.raises(ValueError, match="bfloat16"):
        kq.attention(Q, K, K.half())
    with pytest.raises(ValueError, match="next to each other"):
        kq.attention(Q, K.transpose(0, 2).contiguous().transpose(0, 2), K)
    for bad in (dict(scale=0.0), dict(scale=float("nan"))):
        with pytest.raises(kq.KQError):
            kq.attention(Q, K, K, **bad)
    with pytest.raises(kq.KQError):
        kq.attention(Q[:, :1], K, K)
    with pytest.raises(kq.KQError):                            # strides of whole 16-byte pieces
        kq.attention(torch.zeros(4, 2, 68, dtype=torch.bfloat16, device="cuda")[:, :, :64], K, K)
