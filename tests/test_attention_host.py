"""The 8-bit path's attention without a GPU: the oracle against closed forms, and every refusal of the C ABI
and of the binding."""

import ctypes

import numpy as np
import pytest
import torch

import w4a4_post_quantization_amd as kq
from oracle import attention as oracle

P = ctypes.c_void_p(0x100000)          # 256-byte aligned, never dereferenced: the call is refused first
ODD16 = ctypes.c_void_p(0x100008)
ODD4 = ctypes.c_void_p(0x100002)
NULL, SHAPE, ALIGN, UNSUPPORTED, VALUE, WORKSPACE = 1, 2, 3, 4, 5, 7


@pytest.fixture(scope="module")
def lib():
    return kq.load()


# ---- oracle

def test_oracle_against_torch():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(7, 2, 24)), rng.normal(size=(7, 1, 24)), rng.normal(size=(7, 1, 24))
    for causal in (False, True):
        o, _ = oracle.attention(q, k, v, [0, 7], [0, 7], causal, 0.3, 0.0, 0.0)
        ref = torch.nn.functional.scaled_dot_product_attention(
            *(torch.from_numpy(np.repeat(t, 2 // t.shape[1], axis=1)).transpose(0, 1) for t in (q, k, v)),
            is_causal=causal, scale=0.3).transpose(0, 1).numpy()
        np.testing.assert_allclose(o, ref, rtol=1e-12, atol=1e-13)


def test_oracle_empty_rows_and_shorter_keys():
    rng = np.random.default_rng(1)
    q, k, v = rng.normal(size=(5, 1, 8)), rng.normal(size=(2, 1, 8)), rng.normal(size=(2, 1, 8))
    assert list(oracle.visible(5, 2, True)) == [0, 0, 0, 1, 2]
    o, _ = oracle.attention(q, k, v, [0, 5], [0, 2], True, 1.0, 0.0, 0.0)
    assert np.all(o[:3] == 0)
    np.testing.assert_allclose(o[3, 0], v[0, 0], rtol=1e-15)


def test_oracle_paged_equals_packed():
    rng = np.random.default_rng(2)
    k, v, q = rng.normal(size=(40, 2, 8)), rng.normal(size=(40, 2, 8)), rng.normal(size=(1, 4, 8))
    table = np.array([[2, 0, 3]])
    kc, vc = np.full((4, 2, 16, 8), np.nan), np.full((4, 2, 16, 8), np.nan)
    for j in range(40):
        kc[table[0, j // 16], :, j % 16], vc[table[0, j // 16], :, j % 16] = k[j], v[j]
    a, _ = oracle.paged(q, kc, vc, table, [40], 0.4, 0.0, 0.0)
    b, _ = oracle.attention(q, k, v, [0, 1], [0, 40], True, 0.4, 0.0, 0.0)
    np.testing.assert_allclose(a, b, rtol=1e-13)
    filled = oracle.append(k, np.full_like(kc, np.nan), table, [40], [0, 40], lambda to, new: to.__setitem__(slice(None), new))
    assert np.array_equal(filled, kc, equal_nan=True)


# ---- refusals of the C ABI

def _attention(lib, **kw):
    a = dict(dt=1, Q=P, K=P, V=P, st=(512, 128), kst=(256, 128), vst=(256, 128), cq=P, ck=P, B=2, T=10, Tk=12, Hq=4, Hkv=2,
             D=128, causal=1, scale=0.1, O=P, c=None, s=None, wk=None, nb=0)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.kq_attention(a["dt"], a["Q"], *a["st"], a["K"], *a["kst"], a["V"], *a["vst"], a["cq"], a["ck"], a["B"], a["T"],
                            a["Tk"], a["Hq"], a["Hkv"], a["D"], a["causal"], a["scale"], a["O"], a["c"], a["s"], a["wk"],
                            a["nb"], None)


def _paged(lib, **kw):
    a = dict(dt=1, Q=P, st=(512, 128), k=P, v=P, ks=None, vs=None, pages=9, page=16, table=P, width=4, ln=P, B=3, Hq=4,
             Hkv=2, D=128, scale=0.1, O=P, c=None, s=None, wk=P, nb=1 << 40)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.kq_paged_attention(a["dt"], a["Q"], *a["st"], a["k"], a["v"], a["ks"], a["vs"], a["pages"], a["page"],
                                  a["table"], a["width"], a["ln"], a["B"], a["Hq"], a["Hkv"], a["D"], a["scale"], a["O"],
                                  a["c"], a["s"], a["wk"], a["nb"], None)


def _append(lib, **kw):
    a = dict(dt=1, K=P, V=P, st=(256, 128), vst=(256, 128), cu=P, B=3, T=7, Hkv=2, D=128, table=P, width=4, ln=P, k=P, v=P,
             ks=None, vs=None, pages=9, page=16)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.kq_cache_append(a["dt"], a["K"], *a["st"], a["V"], *a["vst"], a["cu"], a["B"], a["T"], a["Hkv"], a["D"],
                               a["table"], a["width"], a["ln"], a["k"], a["v"], a["ks"], a["vs"], a["pages"], a["page"], None)


def _heads_refusals(call):
    assert call(dt=2) == UNSUPPORTED and call(dt=-1) == UNSUPPORTED
    assert call(D=12) == SHAPE and call(D=0) == SHAPE
    assert call(D=136, st=(1 << 12, 136)) == UNSUPPORTED
    assert call(Hkv=0) == SHAPE


def _output_refusals(call):
    assert call(O=None) == NULL
    assert call(c=P, s=P) == NULL                               # both kinds of output
    assert call(O=None, c=P) == NULL and call(O=None, s=P) == NULL
    assert call(O=None, c=P, s=P, D=64) == UNSUPPORTED
    assert call(O=ODD16) == ALIGN and call(O=None, c=ODD16, s=P) == ALIGN and call(O=None, c=P, s=ODD4) == ALIGN
    for scale in (0.0, -0.1, float("nan"), float("inf"), 3.0e38):
        assert call(scale=scale) == VALUE


def _cache_refusals(call):
    for name in ("k", "v", "table", "ln"):
        assert call(**{name: None}) == NULL
    assert call(ks=P) == NULL and call(vs=P) == NULL            # one without the other
    assert call(ks=P, vs=P, D=72) == SHAPE                      # rows of codes are whole 16-byte pieces
    for bad in (dict(page=8), dict(page=24), dict(page=0), dict(pages=0), dict(width=0)):
        assert call(**bad) == SHAPE
    assert call(page=65552) == UNSUPPORTED and call(width=1 << 27) == UNSUPPORTED and call(pages=1 << 31) == UNSUPPORTED
    for name in ("k", "v"):
        assert call(**{name: ODD16}) == ALIGN
    for name in ("table", "ln"):
        assert call(**{name: ODD4}) == ALIGN
    assert call(ks=ODD16, vs=P) == ALIGN


def test_attention_refusals(lib):
    def call(**kw):
        return _attention(lib, **kw)
    for name in ("Q", "K", "V"):
        assert call(**{name: None}) == NULL
        assert call(**{name: ODD16}) == ALIGN
    assert call(cq=None) == NULL and call(ck=None) == NULL
    assert call(cq=ODD4) == ALIGN and call(ck=ODD4) == ALIGN
    _heads_refusals(call)
    _output_refusals(call)
    assert call(Hq=3) == SHAPE and call(Hq=1) == SHAPE
    for bad in (dict(T=0), dict(Tk=0), dict(B=0), dict(cq=None, ck=None, B=2)):
        assert call(**bad) == SHAPE
    for bad in (dict(T=(1 << 27) + 1), dict(Tk=(1 << 30) + 1), dict(B=(1 << 20) + 1), dict(Hq=8192, Hkv=8192)):
        assert call(**bad) == UNSUPPORTED
    for name in ("st", "kst", "vst"):
        assert call(**{name: (516, 128)}) == SHAPE and call(**{name: (512, 12)}) == SHAPE
        assert call(**{name: (120, 128)}) == SHAPE and call(**{name: (512, -128)}) == SHAPE
        assert call(**{name: ((1 << 21) + 8, 128)}) == UNSUPPORTED


def test_attention_workspace(lib):
    """Few queries of many keys need one; prompts and few keys do not."""
    f = lib.kq_attention_workspace_bytes
    need = f(2, 10, 5000, 1, 4, 2, 128)
    assert need > 0
    assert all(f(B, T, 704, 1, 4, 2, 128) == 0 for B in (1, 2, 7) for T in (1, 10, 100, 1000))     # as the binding relies on
    assert f(1, 8192, 8192, 0, 32, 8, 128) == 0
    assert f(2, 10, 5000, 1, 4, 3, 128) == 0 and f(0, 10, 5000, 1, 4, 2, 128) == 0
    assert _attention(lib, Tk=5000) == WORKSPACE and _attention(lib, Tk=5000, wk=P, nb=need - 1) == WORKSPACE
    assert _attention(lib, Tk=5000, wk=ODD16, nb=need) == ALIGN


def test_paged_refusals(lib):
    def call(**kw):
        return _paged(lib, **kw)
    assert call(Q=None) == NULL and call(Q=ODD16) == ALIGN
    _heads_refusals(call)
    _output_refusals(call)
    _cache_refusals(call)
    assert call(Hq=3) == SHAPE and call(B=0) == SHAPE
    assert call(B=(1 << 20) + 1, width=1) == UNSUPPORTED
    assert call(B=1 << 20, width=1, Hq=16, st=(2048, 128)) == UNSUPPORTED
    assert call(B=1 << 18, width=1 << 16) == UNSUPPORTED        # blocks past 32 bits
    assert call(st=(512, (1 << 21) + 8)) == UNSUPPORTED
    need = lib.kq_paged_attention_workspace_bytes(3, 4, 2, 128, 400, 16)
    assert need > 0 and lib.kq_paged_attention_workspace_bytes(3, 4, 3, 128, 400, 16) == 0
    assert call(width=400, wk=None) == WORKSPACE and call(width=400, nb=need - 1) == WORKSPACE
    assert call(width=400, wk=ODD16) == ALIGN
    assert lib.kq_paged_attention_workspace_bytes(3, 4, 2, 128, 40, 16) == 0          # short tables are not split


def test_append_refusals(lib):
    def call(**kw):
        return _append(lib, **kw)
    assert call(K=None) == NULL and call(V=None) == NULL and call(K=ODD16) == ALIGN and call(V=ODD16) == ALIGN
    assert call(cu=ODD4) == ALIGN
    _heads_refusals(call)
    _cache_refusals(call)
    assert call(T=0) == SHAPE and call(cu=None) == SHAPE and call(B=0) == SHAPE
    assert call(T=(1 << 25) + 1) == UNSUPPORTED
    assert call(st=(120, 128)) == SHAPE and call(vst=(260, 128)) == SHAPE


# ---- refusals of the binding

H = torch.zeros(4, 2, 64, dtype=torch.float16)


def test_binding_refusals():
    with pytest.raises(ValueError, match="3-D"):
        kq.attention(H[0], H, H)
    with pytest.raises(ValueError, match="GPU"):
        kq.attention(H, H, H)
    with pytest.raises(ValueError, match="float16 or torch.bfloat16"):
        kq.attention(H.float(), H, H)
    with pytest.raises(ValueError, match="3-D"):
        kq.cache_append("K", H, H, H, H, H)
    with pytest.raises(ValueError, match="GPU"):
        kq.cache_append(H, H, H, H, H, H)
    with pytest.raises(ValueError, match="GPU"):
        kq.paged_attention(H, H, H, H, H)
