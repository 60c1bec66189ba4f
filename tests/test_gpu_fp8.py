"""GPU parity of the 8-bit path against the float64 oracle.

Tolerances, derived before the first run (u = 2^-24, half a float32 step):
  quantizer   16-bit inputs, a power-of-two scale and one rounding: every byte equal.
  norm        h carries one rounding; the sum of K squares is a chain of at most 8 * 8 fused
              products (then float64), halved by the root; the factor and two products round
              once each: relative error below (1 + 32 + 3) u of y, taken as 64 u.  The residual is one float32 sum rounded once more: equal bits.
  linear      on small whole numbers with small power-of-two scales every partial sum is exact
              in float32, so the output is the exact value rounded once: every bit equal.  On
              random values each of the K additions rounds or truncates at 24 bits: K 2^-23 of
              sum |x w|, plus half a step of the output type.
  gated       gate and up as the linear.  Activation: a handful of roundings, and the argument
              of the exponential carries its own relative error, which the exponential turns
              into |argument| times as much: see ACT_U.
"""

import ctypes

import numpy as np
import pytest
import torch

from oracle import fp8

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


def ACT_U(g, act):
    """Units u of relative error of the float32 activation of an exact g.  For g / (1 + e^-x) an
    error of x moves the result by x sigmoid(-x) of it (x = g for SiLU: one rounding in the
    exponential's argument; x = 2 z for the tanh form, z after five roundings and a cancellation-
    free sum); g erfc(-g / sqrt 2) / 2 is moved by g^2 per unit of its argument where g < 0 and by
    less than one where g > 0.  The library's expf and erfcf are good to a few units."""
    a = np.abs(g)
    if act == "gelu":
        return 32 + np.where(g < 0, 8 * a * a, 0.0)
    x = g if act == "silu" else 1.5957691216 * (g + 0.044715 * g ** 3)
    return 16 + (4 if act == "silu" else 16) * np.abs(x) / (1.0 + np.exp(np.minimum(x, 700.0)))


def _np(t):
    return t.detach().cpu().double().numpy()


def _bytes(t):
    return t.detach().cpu().view(torch.uint8).numpy()


def _act_data(M, K, dtype, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(M, K)) * scale + rng.normal(size=(M, 1))
    x[:, rng.choice(K, size=min(5, K), replace=False)] *= 30.0
    return torch.from_numpy(x).to(DT[dtype])


def _whole(rows, K, seed):
    """Codes of whole numbers -3 .. 3 with scales 2^-1 .. 2^1 (per row and group)."""
    rng = np.random.default_rng(seed)
    codes = fp8.encode(rng.integers(-3, 4, size=(rows, K)).astype(np.float64))
    scales = np.zeros((rows, fp8.scale_cols(K)), np.uint8)
    ng = (K + 127) // 128
    scales[:, :ng] = rng.integers(126, 129, size=(rows, ng))
    return codes, scales


def _dev(codes, scales):
    return torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn), torch.from_numpy(scales).cuda()


def _random_codes(rows, K, seed):
    rng = np.random.default_rng(seed)
    return fp8.quantize(rng.normal(size=(rows, K)) * np.exp(0.3 * rng.normal(size=(rows, 1))))


# ------------------------------------------------------------------------- quantizer

@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (77, 2240), (5, 512), (130, 528), (9, 4096), (2, 16400), (1100, 2064)])
def test_quantize(kq, M, K, dtype):
    x = _act_data(M, K, dtype, M + K)
    codes, scales = kq.quantize_fp8(x.cuda())
    rc, rs = fp8.quantize(_np(x))
    assert np.array_equal(_bytes(scales), rs)
    assert np.array_equal(_bytes(codes), rc)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_quantize_special_values(kq, dtype):
    """Groups of zeros, of subnormals, of the type's extremes, of exact borders (448 2^e and its
    neighbours), and groups that hold an infinity or a NaN beside clean ones."""
    tiny = torch.finfo(DT[dtype]).smallest_normal / 4
    x = torch.zeros(9, 400, dtype=torch.float64)
    x[1] = tiny
    x[2, ::2] = -tiny
    x[3] = torch.finfo(DT[dtype]).max
    x[4, 5], x[4, 130], x[4, 300] = 448.0, 450.0, -896.0
    x[5] = torch.linspace(-3, 3, 400)
    x[5, 17] = float("inf")
    x[6, 399] = float("nan")
    x[7] = -0.0
    x[8] = torch.linspace(-448, 448, 400)
    x = x.to(DT[dtype])
    codes, scales = kq.quantize_fp8(x.cuda())
    rc, rs = fp8.quantize(_np(x))
    assert np.array_equal(_bytes(scales), rs)
    assert np.array_equal(_bytes(codes), rc)
    assert rs[5, 0] == 255 and rs[5, 1] != 255 and rs[6, 3] == 255


def test_outputs_beside_the_rows_are_left_alone(kq):
    x = _act_data(5, 272, "bf16", 3).cuda()
    codes = torch.full((7, 272), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((7, 4), 0x55, dtype=torch.uint8, device="cuda")
    kq.quantize_fp8(x, codes=codes[1:6].view(torch.float8_e4m3fn), scales=scales[1:6])
    for t in (codes, scales):
        assert torch.all(t[0] == 0x55) and torch.all(t[6] == 0x55)
    rc, rs = fp8.quantize(_np(x))
    assert np.array_equal(_bytes(codes[1:6]), rc) and np.array_equal(_bytes(scales[1:6]), rs)


# ------------------------------------------------------------------------- norm

NORM_SHAPES = [(1, 16), (1, 4096), (2, 128), (3, 528), (77, 1152), (5, 2240), (3, 5008), (2, 8192), (2, 11008),
               (1, 16384), (300, 272), (1100, 640), (600, 4096)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("with_residual", [False, True])
@pytest.mark.parametrize("M,K", NORM_SHAPES)
def test_norm(kq, M, K, with_residual, dtype):
    x = _act_data(M, K, dtype, 7 * M + K)
    r = _act_data(M, K, dtype, 7 * M + K + 1, 3.0) if with_residual else None
    rng = np.random.default_rng(K)
    gamma = torch.from_numpy(1.0 + 0.3 * rng.normal(size=K)).to(DT[dtype])
    codes, scales, out = kq.rmsnorm_quantize_fp8(x.cuda(), gamma.cuda(), eps=1e-5,
                                                 residual=None if r is None else r.cuda())
    h, y = fp8.rmsnorm(_np(x), None if r is None else _np(r), _np(gamma), float(np.float32(1e-5)))
    errors = fp8.check_codes(_bytes(codes), _bytes(scales), y, 64 * U * np.abs(y))
    assert not errors, errors[:5]
    if with_residual:
        ref = (x.float() + r.float()).to(DT[dtype])
        assert torch.equal(out.cpu(), ref)
    else:
        assert out is None


def test_norm_residual_in_place(kq):
    x, r = _act_data(33, 1152, "bf16", 1).cuda(), _act_data(33, 1152, "bf16", 2).cuda()
    gamma = torch.ones(1152, dtype=torch.bfloat16, device="cuda")
    c0, s0, out = kq.rmsnorm_quantize_fp8(x, gamma, residual=r)
    h = r.clone()
    c1, s1, h1 = kq.rmsnorm_quantize_fp8(x, gamma, residual=h, residual_out=h)
    assert h1 is h and torch.equal(h, out)
    assert torch.equal(c0.view(torch.uint8), c1.view(torch.uint8)) and torch.equal(s0, s1)


def test_norm_more_rows_than_a_grid(kq):
    """More rows than workgroups: every row of the last turn is there."""
    M, K = (1 << 22) + 1000, 32
    x = torch.ones(M, K, dtype=torch.float16, device="cuda")
    tail = _act_data(1003, K, "fp16", 6)
    x[-1003:] = tail.cuda()
    gamma = torch.full((K,), 0.5, dtype=torch.float16, device="cuda")
    codes, scales, _ = kq.rmsnorm_quantize_fp8(x, gamma)
    _, y = fp8.rmsnorm(_np(tail), None, np.full(K, 0.5), float(np.float32(1e-6)))
    assert not fp8.check_codes(_bytes(codes[-1003:]), _bytes(scales[-1003:]), y, 64 * U * np.abs(y))
    # rows of ones: 0.5 / sqrt(1 + 1e-6) is 256 2^-9 to within a code
    assert torch.all(codes[:-1003].view(torch.uint8) == 0x78) and torch.all(scales[:-1003, 0] == 127 - 9)


def test_norm_special_rows(kq):
    """A row of zeros gives zeros (eps > 0); a row with a NaN is NaN throughout; in a row with an
    infinity that value's group is NaN and the other groups are zero."""
    x = _act_data(4, 512, "bf16", 5)
    x[0] = 0
    x[1, 200] = float("nan")
    x[2, 300] = float("-inf")
    gamma = torch.ones(512, dtype=torch.bfloat16)
    codes, scales, _ = kq.rmsnorm_quantize_fp8(x.cuda(), gamma.cuda())
    codes, scales = _bytes(codes), _bytes(scales)
    assert not codes[0].any() and not scales[0].any()
    assert np.all(codes[1] == 0x7F) and np.all(scales[1] == 255)
    assert scales[2].tolist() == [0, 0, 255, 0] and np.all(codes[2, 256:384] == 0x7F)
    assert not (codes[2, :256] & 0x7F).any() and not (codes[2, 384:] & 0x7F).any()
    _, y = fp8.rmsnorm(_np(x[3:]), None, _np(gamma), 1e-6)
    assert not fp8.check_codes(codes[3:], scales[3:], y, 64 * U * np.abs(y))


# ------------------------------------------------------------------------- linear

LINEAR_SHAPES = [
    (1, 16, 16), (1, 16, 48), (1, 128, 4096), (1, 4096, 1152), (2, 144, 528), (3, 272, 2240), (5, 1152, 1152),
    (8, 2064, 640), (15, 48, 11008), (16, 512, 1024), (17, 528, 1040), (31, 64, 144), (32, 1024, 512), (33, 80, 272),
    (37, 6144, 512), (48, 272, 912), (63, 400, 2240), (64, 640, 128), (65, 272, 256), (96, 1152, 4096), (100, 2240, 5600),
    (128, 256, 1024), (129, 272, 128), (200, 144, 2240), (255, 256, 64), (256, 512, 512), (257, 784, 400),
    (300, 1152, 1152), (513, 528, 272), (1000, 2240, 1152), (1024, 1024, 1024), (1025, 4112, 16), (2060, 1552, 640),
    (5, 272, 16400), (40, 48, 33040),                                  # more than one set of scale bytes
    (1031, 4112, 4304), (4100, 4112, 272), (2500, 8208, 656), (1290, 6160, 144),   # large tiles, whole and halved
]


def _linear_case(kq, M, N, K, dtype, bias, seed=0):
    xc, xs = _whole(M, K, seed + M)
    wc, ws = _whole(N, K, seed + N + 1)
    b = torch.from_numpy(np.random.default_rng(seed).integers(-9, 10, size=N).astype(np.float64)).to(DT[dtype])
    Y = kq.fp8_linear(*_dev(xc, xs), *_dev(wc, ws), bias=b.cuda() if bias else None, dtype=DT[dtype])
    ref = fp8.dequantize(xc, xs) @ fp8.dequantize(wc, ws).T
    if bias:
        ref = ref + _np(b)
    return Y.cpu(), torch.from_numpy(ref).to(DT[dtype])


@pytest.mark.parametrize("M,N,K", LINEAR_SHAPES)
def test_linear_exact(kq, M, N, K):
    """Every output, bit for bit: a lost or doubled product, a wrong scale or a wrong row shows."""
    dtype, bias = ("bf16", M % 2 == 0) if (M + N // 16) % 2 else ("fp16", M % 2 == 1)
    got, ref = _linear_case(kq, M, N, K, dtype, bias)
    assert torch.equal(got, ref), (got - ref).abs().max()


@pytest.mark.parametrize("M", [1, 16, 30, 45, 61])
@pytest.mark.parametrize("N,K", [(2048, 528), (4096, 6160), (4112, 528), (4112, 6160), (8192, 144), (8208, 528)])
def test_linear_few_tokens_exact(kq, M, N, K):
    """Up to 64 tokens, to each side of one and two workgroups of 16 weight rows on a compute unit."""
    got, ref = _linear_case(kq, M, N, K, "fp16", M % 2 == 0, seed=M + N)
    assert torch.equal(got, ref)


@pytest.mark.parametrize("M,N,K", [(4100, 4368, 144), (4100, 4368, 256), (9000, 2304, 528), (4352, 4352, 2048), (3850, 5136, 2064),
                                   (4096, 8736, 2176), (4352, 4352, 4096), (4352, 4352, 4112)])
def test_many_tiles_exact(kq, M, N, K):
    """More whole tiles than compute units: sequences of tiles on a workgroup, of 2 to 33 stages, and behind them the
    tiles of fewer tokens; the same codes as a gated pair where N is even in 32s."""
    g = torch.Generator(device="cuda").manual_seed(M + K)
    ng = (K + 127) // 128

    def whole(rows, low):
        c = torch.randint(-3, 4, (rows, K), device="cuda", generator=g).float().to(torch.float8_e4m3fn)
        s = torch.zeros(rows, kq.fp8_scale_cols(K), dtype=torch.uint8, device="cuda")
        s[:, :ng] = torch.randint(low, low + 3, (rows, ng), device="cuda", generator=g, dtype=torch.uint8)
        return c, s

    def value(c, s):
        unit = torch.exp2(torch.arange(256, device="cuda", dtype=torch.float64) - 127)[s[:, :(c.shape[1] + 127) // 128].long()]
        return c.double() * unit.repeat_interleave(128, 1)[:, :c.shape[1]]

    w, ws = whole(N, 126)
    x, xs = whole(M, 126)
    bias = torch.randint(-9, 10, (N,), device="cuda", generator=g).to(torch.bfloat16)
    ref = (value(x, xs) @ value(w, ws).t() + bias.double()).float().to(torch.bfloat16)      # sums exact in float32
    assert torch.equal(kq.fp8_linear(x, xs, w, ws, bias=bias, dtype=torch.bfloat16), ref)
    if N % 32:
        return
    F = N // 2
    x, xs = whole(M, 120)
    codes, scales = kq.fp8_gated_linear(x, xs, w, ws, act="silu")
    y = value(x, xs) @ value(w, ws).t()
    h = y[:, :F] * torch.sigmoid(y[:, :F]) * y[:, F:]
    G = (F + 127) // 128
    top = torch.nn.functional.pad(h, (0, 128 * G - F)).view(M, G, 128).abs().amax(2)
    unit = torch.exp2(torch.arange(256, device="cuda", dtype=torch.float64) - 127)[scales[:, :G].long()]
    # the scale is the smallest without saturation, a code within half a step of E4M3 (2^-4 relative,
    # 2^-10 of the unit below its normal numbers); 1e-4 for the float32 activation
    assert bool(((top <= 448 * unit * (1 + 1e-4)) & ((top >= 224 * unit * (1 - 1e-4)) | (top == 0))).all())
    err, step = (value(codes, scales) - h).abs(), torch.maximum(h.abs() * 2.0 ** -4, unit.repeat_interleave(128, 1)[:, :F] * 2.0 ** -10)
    assert bool((err <= step + 1e-4 * h.abs() + 1e-30).all())


@pytest.mark.parametrize("M", list(range(1, 20)) + [24, 40, 56, 72, 88, 112, 144, 160, 192, 224])
def test_linear_rows(kq, M):
    got, ref = _linear_case(kq, M, 208, 656, "bf16", True, seed=3)
    assert torch.equal(got, ref)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 512, 4096), (7, 272, 2240), (50, 1040, 1152), (160, 528, 4096), (700, 784, 1552)])
def test_linear_random(kq, M, N, K, dtype):
    xc, xs = _random_codes(M, K, M)
    wc, ws = _random_codes(N, K, N)
    Y = _np(kq.fp8_linear(*_dev(xc, xs), *_dev(wc, ws), dtype=DT[dtype]))
    x, w = fp8.dequantize(xc, xs), fp8.dequantize(wc, ws)
    ref = x @ w.T
    tol = torch.finfo(DT[dtype]).eps / 2 * np.abs(ref) * (1 + 1e-6) + K * 2.0 ** -23 * (np.abs(x) @ np.abs(w).T) + 2.0 ** -25
    assert np.all(np.abs(Y - ref) <= tol), np.max(np.abs(Y - ref) / tol)


@pytest.mark.parametrize("M", [1, 20, 100, 400])
def test_linear_nan_and_overflow(kq, M):
    """A NaN group makes NaN exactly the outputs that use it; a sum past the type is infinite."""
    N, K = 272, 400
    xc, xs = _whole(M, K, 1)
    wc, ws = _whole(N, K, 2)
    xc[M - 1, 256:384], xs[M - 1, 2] = 0x7F, 255
    wc[33, 384:], ws[33, 3] = 0x7F, 255
    xs[0, 0], ws[5, 0] = 127 + 20, 127 + 20
    Y = kq.fp8_linear(*_dev(xc, xs), *_dev(wc, ws), dtype=torch.float16).cpu()
    ref = torch.from_numpy(fp8.dequantize(xc, xs) @ fp8.dequantize(wc, ws).T)
    assert torch.equal(torch.isnan(Y), torch.isnan(ref))
    assert torch.isnan(Y[M - 1]).all() and torch.isnan(Y[:, 33]).all()
    fine = ~torch.isnan(ref)
    ref16 = ref.to(torch.float16)
    ok = fine & (ref.abs() < 2.0 ** 15)
    ok[0], ok[:, 5] = False, False                 # their small terms need more than 24 bits
    assert torch.equal(Y[ok], ref16[ok])
    over = fine & (ref.abs() > 65520 * 1.01)
    if M > 1:
        assert over.any()
    assert torch.equal(Y[over], ref16[over])


def test_linear_extreme_scales(kq):
    """Scale bytes at both ends: 2^-127 times 2^100 and back, in range of the output."""
    K, N = 256, 64
    for M in (3, 300):
        xc, xs = _whole(M, K, 4)
        wc, ws = _whole(N, K, 5)
        xs[:, :2], ws[:, :2] = 1, 253
        Y = kq.fp8_linear(*_dev(xc, xs), *_dev(wc, ws), dtype=torch.bfloat16).cpu()
        assert torch.equal(Y, torch.from_numpy(fp8.dequantize(xc, xs) @ fp8.dequantize(wc, ws).T).to(torch.bfloat16))


# ------------------------------------------------------------------------- gated

GATED_SHAPES = [(1, 16, 16), (1, 128, 4096), (1, 1152, 512), (2, 144, 528), (3, 272, 272), (7, 2240, 1152), (16, 400, 1040),
                (17, 528, 640), (32, 1024, 256), (33, 144, 144), (64, 256, 2240), (65, 272, 528), (100, 640, 1152),
                (128, 128, 512), (130, 144, 400), (203, 1104, 2240), (256, 256, 1024), (300, 528, 272), (513, 1152, 640),
                (1030, 784, 528), (2050, 272, 128),
                (3, 48, 16400), (40, 144, 16656), (1030, 2064, 528), (2050, 4112, 400), (600, 11024, 272),
                (1100, 2192, 4240), (30, 12304, 144), (45, 12288, 144), (48, 12304, 272), (60, 8192, 144), (49, 8208, 272)]


@pytest.mark.parametrize("M,F,K", GATED_SHAPES)
def test_gated(kq, M, F, K):
    act = ["silu", "gelu", "gelu_tanh"][(M + F // 16 + K // 16) % 3]
    xc, xs = _whole(M, K, M)
    wc, ws = _whole(2 * F, K, F)
    # products of about unit size: exact gate and up, no overflow in the product
    xs[:, : (K + 127) // 128] -= 6
    codes, scales = kq.fp8_gated_linear(*_dev(xc, xs), *_dev(wc, ws), act=act)
    g, u, h = fp8.gated(xc, xs, wc, ws, act)
    tau = np.abs(h) * U * (ACT_U(g, act) + 2) + 2.0 ** -140
    errors = fp8.check_codes(_bytes(codes), _bytes(scales), h, tau)
    assert not errors, errors[:5]


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M", [1, 40, 260])
def test_gated_random(kq, M, act):
    F, K = 272, 1040
    xc, xs = _random_codes(M, K, M)
    wc, ws = fp8.quantize(np.random.default_rng(9).normal(size=(2 * F, K)) / np.sqrt(K) * 2)
    codes, scales = kq.fp8_gated_linear(*_dev(xc, xs), *_dev(wc, ws), act=act)
    g, u, h = fp8.gated(xc, xs, wc, ws, act)
    d = K * 2.0 ** -23 * (np.abs(fp8.dequantize(xc, xs)) @ np.abs(fp8.dequantize(wc, ws)).T)
    dg, du = d[:, :F], d[:, F:]
    # |act'| <= 1.13 for the three activations
    tau = np.abs(h) * U * (ACT_U(g, act) + 2) + 1.13 * dg * np.abs(u) + (np.abs(fp8.activation(g, act)) + 1.13 * dg) * du
    errors = fp8.check_codes(_bytes(codes), _bytes(scales), h, tau)
    assert not errors, errors[:5]


@pytest.mark.parametrize("M", [1, 40, 300])
def test_gated_large_gates_and_nan(kq, M):
    """Gates far out on both sides (the exponential over- and underflows) stay finite; a NaN
    token makes its own groups NaN and no others."""
    F, K = 144, 128
    xc, xs = _whole(M, K, 1)
    wc, ws = _whole(2 * F, K, 2)
    xs[:, 0] += 6
    if M > 1:
        xc[M // 2], xs[M // 2, 0] = 0x7F, 255
    for act in ("silu", "gelu", "gelu_tanh"):
        codes, scales = kq.fp8_gated_linear(*_dev(xc, xs), *_dev(wc, ws), act=act)
        codes, scales = _bytes(codes), _bytes(scales)
        keep = np.arange(M) != (M // 2 if M > 1 else -1)
        with np.errstate(over="ignore", under="ignore"):
            g, u, h = fp8.gated(xc[keep], xs[keep], wc, ws, act)
        tau = np.abs(h) * U * (ACT_U(g, act) + 2) + np.abs(u) * 2.0 ** -100
        errors = fp8.check_codes(codes[keep], scales[keep], h, tau)
        assert not errors, (act, errors[:5])
        if M > 1:
            assert np.all(codes[M // 2] == 0x7F) and np.all(scales[M // 2, :2] == 255)


# ------------------------------------------------------------------------- together, and around

def _block_weights(kq, D, F, seed):
    rng = np.random.default_rng(seed)
    gu = torch.from_numpy(rng.normal(size=(2 * F, D)) / np.sqrt(D)).to(torch.bfloat16).cuda()
    dn = torch.from_numpy(rng.normal(size=(D, F)) / np.sqrt(F)).to(torch.bfloat16).cuda()
    gamma = torch.from_numpy(1 + 0.1 * rng.normal(size=D)).to(torch.bfloat16).cuda()
    return kq.quantize_fp8(gu), kq.quantize_fp8(dn), gamma


def _block(kq, x, h, w, stream=None):
    (guc, gus), (dc, ds), gamma = w
    c1, s1, h1 = kq.rmsnorm_quantize_fp8(x, gamma, residual=h, stream=stream)
    c2, s2 = kq.fp8_gated_linear(c1, s1, guc, gus, act="silu", stream=stream)
    y = kq.fp8_linear(c2, s2, dc, ds, dtype=torch.bfloat16, stream=stream)
    c3, s3, h2 = kq.rmsnorm_quantize_fp8(y, gamma, residual=h1, stream=stream)
    return c1, s1, c2, s2, y, c3, s3, h2


@pytest.mark.parametrize("M", [1, 45, 333])
def test_feed_forward_block(kq, M):
    """Norm, gate and up, down, next norm: each stage against the oracle on the codes that the
    stage before it produced."""
    D, F = 640, 1104
    w = _block_weights(kq, D, F, 1)
    x, h = _act_data(M, D, "bf16", 11), _act_data(M, D, "bf16", 12)
    c1, s1, c2, s2, y, c3, s3, h2 = _block(kq, x.cuda(), h.cuda(), w)
    (guc, gus), (dc, ds), gamma = w
    h1, n1 = fp8.rmsnorm(_np(x), _np(h), _np(gamma), float(np.float32(1e-6)))
    assert not fp8.check_codes(_bytes(c1), _bytes(s1), n1, 64 * U * np.abs(n1))
    g, u, a = fp8.gated(_bytes(c1), _bytes(s1), _bytes(guc), _bytes(gus), "silu")
    d = D * 2.0 ** -23 * (np.abs(fp8.dequantize(_bytes(c1), _bytes(s1))) @ np.abs(fp8.dequantize(_bytes(guc), _bytes(gus))).T)
    tau = np.abs(a) * U * (ACT_U(g, "silu") + 2) + 1.13 * d[:, :F] * np.abs(u) + (np.abs(fp8.activation(g, "silu")) + 1.13 * d[:, :F]) * d[:, F:]
    assert not fp8.check_codes(_bytes(c2), _bytes(s2), a, tau)
    xa, wa = fp8.dequantize(_bytes(c2), _bytes(s2)), fp8.dequantize(_bytes(dc), _bytes(ds))
    ref = xa @ wa.T
    tol = 2.0 ** -8 * np.abs(ref) * (1 + 1e-6) + F * 2.0 ** -23 * (np.abs(xa) @ np.abs(wa).T)
    assert np.all(np.abs(_np(y) - ref) <= tol)
    hr = (x.float() + h.float()).to(torch.bfloat16)
    assert torch.equal(h2.cpu(), (y.cpu().float() + hr.float()).to(torch.bfloat16))


@pytest.mark.parametrize("M", [1, 24, 150])
def test_block_same_bits_every_time_and_on_another_stream(kq, M):
    w = _block_weights(kq, 512, 2064, 2)
    x, h = _act_data(M, 512, "bf16", 1).cuda(), _act_data(M, 512, "bf16", 2).cuda()
    first = _block(kq, x, h, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    runs = [_block(kq, x, h, w), _block(kq, x, h, w, stream=side)]
    torch.cuda.synchronize()
    for r in runs:
        for a, b in zip(first, r):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_two_blocks_at_once(kq):
    """Two blocks in flight on two streams, each with its own workspaces, do not disturb each
    other."""
    w = _block_weights(kq, 512, 2064, 2)
    args = [(_act_data(9 + k, 512, "bf16", k).cuda(), _act_data(9 + k, 512, "bf16", 20 + k).cuda()) for k in range(2)]
    refs = [_block(kq, *a, w) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        outs = [_block(kq, *a, w, stream=s) for a, s in zip(args, streams)]
        torch.cuda.synchronize()
        for ref, out in zip(refs, outs):
            for a, b in zip(ref, out):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("M", [1, 70, 300])
def test_block_captured_and_replayed(kq, M):
    """A captured block replayed on new inputs, with eager work and waits between, gives the
    eager block's bytes each time."""
    w = _block_weights(kq, 512, 1104, 3)
    x, h = _act_data(M, 512, "bf16", 1).cuda(), _act_data(M, 512, "bf16", 2).cuda()
    _block(kq, x, h, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _block(kq, x, h, w)
    for k in range(4):
        x.copy_(_act_data(M, 512, "bf16", 50 + k).cuda())
        h.copy_(_act_data(M, 512, "bf16", 90 + k).cuda())
        graph.replay()
        torch.cuda.synchronize()
        ref = _block(kq, x, h, w)
        torch.cuda.synchronize()
        for a, b in zip(out, ref):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), k


def test_rows_do_not_depend_on_the_batch_or_its_padding(kq):
    """Rows behind the last token are not read: NaN there changes nothing before them."""
    K, N = 656, 272
    xc, xs = _whole(70, K, 1)
    wc, ws = _whole(N, K, 2)
    clean = kq.fp8_linear(*_dev(xc[:41], xs[:41]), *_dev(wc, ws), dtype=torch.bfloat16)
    xc[41:], xs[41:] = 0x7F, 255
    c, s = _dev(xc, xs)
    Y = torch.full((70, N), 7.0, dtype=torch.bfloat16, device="cuda")
    kq.fp8_linear(c[:41], s[:41], *_dev(wc, ws), Y=Y[:41])
    assert torch.equal(Y[:41], clean) and torch.all(Y[41:] == 7.0)


def test_offsets_past_32_bits(kq):
    """Arrays of more than 2^31 values and 2^32 bytes: the last rows come out right."""
    K = 16384
    M = (1 << 31) // K + 5
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    tail = _act_data(3, K, "bf16", 8)
    x[-3:] = tail.cuda()
    codes, scales = kq.quantize_fp8(x)
    rc, rs = fp8.quantize(_np(tail))
    assert np.array_equal(_bytes(codes[-3:]), rc) and np.array_equal(_bytes(scales[-3:]), rs)
    assert not codes[: M - 3].view(torch.uint8).any()
    gamma = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    c2, s2, _ = kq.rmsnorm_quantize_fp8(x, gamma, codes=codes, scales=scales)
    _, y = fp8.rmsnorm(_np(tail), None, np.ones(K), 1e-6)
    assert not fp8.check_codes(_bytes(c2[-3:]), _bytes(s2[-3:]), y, 64 * U * np.abs(y))
    del x, c2, s2
    # the codes as activations [M][K] and as weights [N][K], then an output of more than 2^31 values
    wc, ws = _whole(32, K, 5)
    xc, xs = _whole(3, K, 6)
    codes[-3:] = _dev(xc, xs)[0]
    scales[-3:] = _dev(xc, xs)[1]
    ref = torch.from_numpy(fp8.dequantize(xc, xs) @ fp8.dequantize(wc, ws).T).to(torch.float16)
    Y = kq.fp8_linear(codes, scales, *_dev(wc, ws))
    assert torch.equal(Y[-3:].cpu(), ref)
    n = M - M % 16
    Yt = kq.fp8_linear(*_dev(wc[:2], ws[:2]), codes[-n:], scales[-n:])
    assert torch.equal(Yt[:, -3:].cpu(), ref.t()[:2])
    del codes, scales, Y, Yt
    N = 16384
    xc, xs = _whole(5, 16, 9)
    wc, ws = _whole(N, 16, 10)
    big = torch.zeros(M, 16, dtype=torch.uint8, device="cuda")
    bs = torch.zeros(M, 4, dtype=torch.uint8, device="cuda")
    big[-5:], bs[-5:] = torch.from_numpy(xc).cuda(), torch.from_numpy(xs).cuda()
    Y = kq.fp8_linear(big.view(torch.float8_e4m3fn), bs, *_dev(wc, ws))
    ref = torch.from_numpy(fp8.dequantize(xc, xs) @ fp8.dequantize(wc, ws).T).to(torch.float16)
    assert torch.equal(Y[-5:].cpu(), ref)


def test_given_workspace_and_refusals(kq):
    xc, xs = _whole(40, 512, 1)
    wc, ws = _whole(64, 512, 2)
    a, b = _dev(xc, xs), _dev(wc, ws)
    need = kq.fp8_gated_linear_workspace_bytes(40, 32, 512)
    ref = kq.fp8_gated_linear(*a, *b)
    got = kq.fp8_gated_linear(*a, *b, workspace=torch.empty(need + 256, dtype=torch.uint8, device="cuda"))
    assert torch.equal(ref[0].view(torch.uint8), got[0].view(torch.uint8)) and torch.equal(ref[1], got[1])
    if need:
        with pytest.raises(kq.KQError):
            kq.fp8_gated_linear(*a, *b, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        kq.fp8_linear(a[0], a[1][:, :2], *b)                       # scale columns
    with pytest.raises(ValueError):
        kq.fp8_linear(*a, b[0][:, :256], b[1])                     # K
    with pytest.raises(ValueError):
        kq.fp8_linear(*a, *b, bias=torch.zeros(64, device="cuda"))     # float32 bias
    with pytest.raises(ValueError):
        kq.fp8_linear(a[0].t().contiguous().t(), a[1], *b)         # not contiguous
    with pytest.raises(kq.KQError):
        kq.fp8_linear(*a, b[0][:40], b[1][:40])                    # N not a multiple of 16
    x = torch.zeros(4, 40, dtype=torch.float16, device="cuda")
    with pytest.raises(kq.KQError):
        kq.quantize_fp8(x)                                         # K not a multiple of 16
    with pytest.raises(kq.KQError):
        kq.rmsnorm_quantize_fp8(torch.zeros(1, 16400, dtype=torch.float16, device="cuda"),
                                torch.zeros(16400, dtype=torch.float16, device="cuda"))
