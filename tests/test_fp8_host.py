"""The 8-bit path without a GPU: the oracle against torch's conversions and closed forms, and
every refusal of the C ABI and of the binding."""

import ctypes

import numpy as np
import pytest
import torch

import w4a4_post_quantization_amd as kq
from oracle import fp8

P = ctypes.c_void_p(0x100000)          # 256-byte aligned, never dereferenced: the call is refused first
ODD16 = ctypes.c_void_p(0x100008)
ODD4 = ctypes.c_void_p(0x100002)
NULL, SHAPE, ALIGN, UNSUPPORTED, VALUE, WORKSPACE = 1, 2, 3, 4, 5, 7


@pytest.fixture(scope="module")
def lib():
    return kq.load()


# ---- oracle

def test_values_match_torch():
    got = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, fp8.VALUES, equal_nan=True)


def test_encode_matches_torch_with_ties():
    mids = np.concatenate([fp8.MIDPOINTS, fp8.MAGNITUDES, fp8.MIDPOINTS * (1 + 2.0 ** -20), fp8.MIDPOINTS * (1 - 2.0 ** -20)])
    rng = np.random.default_rng(0)
    v = np.concatenate([mids, rng.uniform(-448, 448, 4000), rng.normal(0, 2.0 ** -7, 4000)])
    v = np.concatenate([v, -v]).astype(np.float32)
    v = v[np.abs(v) <= 448.0]
    ref = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fp8.encode(v.astype(np.float64)), ref)


def test_scale_exponent_borders():
    for e in (-30, -1, 0, 7):
        top = 448.0 * 2.0 ** e
        assert fp8.scale_exponent(top) == e
        assert fp8.scale_exponent(np.nextafter(top, np.inf)) == e + 1
        assert fp8.scale_exponent(np.nextafter(top / 2, np.inf)) == e
    assert fp8.scale_exponent(0.0) == -127
    assert fp8.scale_exponent(2.0 ** -140) == -127


def test_quantize_round_trip_error():
    rng = np.random.default_rng(1)
    y = rng.normal(size=(5, 300)) * np.exp(rng.normal(size=(5, 1)))
    codes, scales = fp8.quantize(y)
    back = fp8.dequantize(codes, scales)
    unit = np.ldexp(1.0, np.repeat(scales.astype(int) - 127, 128, axis=1)[:, :300])
    # half a step: 2^-4 of the value, or half of the smallest subnormal
    assert np.all(np.abs(back - y) <= np.maximum(np.abs(y) * 2.0 ** -4, unit * 2.0 ** -10))
    assert not fp8.check_codes(codes, scales, y, np.zeros_like(y))


def test_check_codes_sees_planted_mistakes():
    rng = np.random.default_rng(2)
    y = rng.normal(size=(3, 200))
    codes, scales = fp8.quantize(y)
    tau = np.abs(y) * 1e-6
    for at, change in (((1, 7), 1), ((2, 199), 0x80)):
        c = codes.copy()
        c[at] ^= change
        assert fp8.check_codes(c, scales, y, tau)
    s = scales.copy()
    s[0, 1] += 1
    assert fp8.check_codes(codes, s, y, tau)
    s = scales.copy()
    s[0, 3] = 1                                             # padding
    assert fp8.check_codes(codes, s, y, tau)


# ---- refusals

def test_scale_cols(lib):
    for K, n in ((16, 4), (512, 4), (528, 8), (2240, 20), (1 << 20, 8192)):
        assert lib.kq_fp8_scale_cols(K) == n == kq.fp8_scale_cols(K)
    assert lib.kq_fp8_scale_cols(0) == 0 and lib.kq_fp8_scale_cols((1 << 20) + 16) == 0


def test_quantize_refusals(lib):
    f = lib.kq_quantize_fp8
    assert f(0, None, 4, 64, P, P, None) == NULL
    assert f(0, P, 4, 64, None, P, None) == NULL
    assert f(0, P, 4, 64, P, None, None) == NULL
    assert f(2, P, 4, 64, P, P, None) == UNSUPPORTED
    assert f(0, P, 0, 64, P, P, None) == SHAPE
    assert f(0, P, 4, 0, P, P, None) == SHAPE
    assert f(0, P, 4, 72, P, P, None) == SHAPE
    assert f(0, P, (1 << 30) + 1, 64, P, P, None) == UNSUPPORTED
    assert f(0, P, 4, (1 << 20) + 16, P, P, None) == UNSUPPORTED
    assert f(0, ODD16, 4, 64, P, P, None) == ALIGN
    assert f(0, P, 4, 64, ODD16, P, None) == ALIGN
    assert f(0, P, 4, 64, P, ODD4, None) == ALIGN


def test_norm_refusals(lib):
    f = lib.kq_rmsnorm_quantize_fp8
    ok = dict(dt=1, X=P, r=P, g=P, eps=1e-6, M=4, K=64, c=P, s=P, o=P)

    def call(**kw):
        a = {**ok, **kw}
        return f(a["dt"], a["X"], a["r"], a["g"], a["eps"], a["M"], a["K"], a["c"], a["s"], a["o"], None)
    for name in ("X", "g", "c", "s", "o"):
        assert call(**{name: None}) == NULL
    assert call(dt=-1) == UNSUPPORTED
    assert call(M=0) == SHAPE and call(K=40) == SHAPE
    assert call(K=16384 + 16) == UNSUPPORTED
    for eps in (-1e-6, float("nan"), float("inf")):
        assert call(eps=eps) == VALUE
    for name in ("X", "r", "g", "c", "o"):
        assert call(**{name: ODD16}) == ALIGN
    assert call(s=ODD4) == ALIGN


def test_linear_refusals(lib):
    f = lib.kq_fp8_linear
    ok = dict(dt=1, x=P, xs=P, M=4, K=64, w=P, ws=P, N=32, b=P, Y=P)

    def call(**kw):
        a = {**ok, **kw}
        return f(a["dt"], a["x"], a["xs"], a["M"], a["K"], a["w"], a["ws"], a["N"], a["b"], a["Y"], None)
    for name in ("x", "xs", "w", "ws", "Y"):
        assert call(**{name: None}) == NULL
    assert call(dt=2) == UNSUPPORTED
    assert call(M=0) == SHAPE and call(K=24) == SHAPE and call(N=40) == SHAPE and call(N=0) == SHAPE
    assert call(M=(1 << 30) + 1) == UNSUPPORTED and call(N=(1 << 20) + 16) == UNSUPPORTED
    for name in ("x", "w", "Y", "b"):
        assert call(**{name: ODD16}) == ALIGN
    for name in ("xs", "ws"):
        assert call(**{name: ODD4}) == ALIGN


def test_gated_refusals(lib):
    f = lib.kq_fp8_gated_linear
    ok = dict(act=0, x=P, xs=P, M=4, K=64, w=P, ws=P, F=32, c=P, s=P, wk=P, nb=1 << 40)

    def call(**kw):
        a = {**ok, **kw}
        return f(a["act"], a["x"], a["xs"], a["M"], a["K"], a["w"], a["ws"], a["F"], a["c"], a["s"], a["wk"], a["nb"], None)
    for name in ("x", "xs", "w", "ws", "c", "s"):
        assert call(**{name: None}) == NULL
    assert call(act=3) == UNSUPPORTED and call(act=-1) == UNSUPPORTED
    assert call(M=0) == SHAPE and call(K=24) == SHAPE and call(F=40) == SHAPE
    assert call(F=(1 << 19) + 16) == UNSUPPORTED
    for name in ("x", "w", "c"):
        assert call(**{name: ODD16}) == ALIGN
    for name in ("xs", "ws", "s"):
        assert call(**{name: ODD4}) == ALIGN
    need = lib.kq_fp8_gated_linear_workspace_bytes(4, 32, 64)
    if need:
        assert call(wk=None, nb=0) == WORKSPACE
        assert call(nb=need - 1) == WORKSPACE
        assert call(wk=ODD16) == ALIGN
    assert lib.kq_fp8_gated_linear_workspace_bytes(4, 40, 64) == 0


def test_binding_refuses_host_and_wrong_tensors():
    x = torch.zeros(4, 64, dtype=torch.float16)
    c, s = torch.zeros(4, 64, dtype=torch.float8_e4m3fn), torch.zeros(4, 4, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        kq.quantize_fp8(x)
    with pytest.raises(ValueError, match="float16 or torch.bfloat16"):
        kq.quantize_fp8(x.float())
    with pytest.raises(ValueError, match="2-D"):
        kq.quantize_fp8(x[0])
    with pytest.raises(ValueError, match="GPU"):
        kq.rmsnorm_quantize_fp8(x, x[0])
    with pytest.raises(ValueError, match="GPU"):
        kq.fp8_linear(c, s, c, s)
    with pytest.raises(ValueError, match="act must be"):
        kq.fp8_gated_linear(c, s, c, s, act="relu")
