"""Oracle of the 8-bit path in float64: E4M3 with one E8M0 scale per 128 consecutive values.

E4M3 (OCP 8-bit floating point): sign, 4 exponent bits (bias 7), 3 mantissa bits; code
0x7F / 0xFF is NaN, no infinities, largest 448, subnormals down to 2^-9.  Codes are found by
search over the table of all values, not by a conversion routine.
"""

import math

import numpy as np

GROUP = 128
MAX = 448.0


def _magnitudes():
    v = []
    for b in range(0x7F):
        e, m = b >> 3, b & 7
        v.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(v)


MAGNITUDES = _magnitudes()                    # value of code b = 0 .. 0x7E (ascending)
VALUES = np.concatenate([MAGNITUDES, [np.nan], -MAGNITUDES, [np.nan]])
MIDPOINTS = 0.5 * (MAGNITUDES[1:] + MAGNITUDES[:-1])      # exact in float64


def scale_cols(K):
    return 4 * ((K + 511) // 512)


def encode(v):
    """E4M3 code of each |v| <= 448 (round to nearest, ties to the even code)."""
    a = np.abs(v)
    lo = np.searchsorted(MIDPOINTS, a, side="left")       # a tie gives the lower neighbour
    tie = (lo < len(MIDPOINTS)) & (a == MIDPOINTS[np.minimum(lo, len(MIDPOINTS) - 1)])
    code = np.where(tie & (lo % 2 == 1), lo + 1, lo)
    return (code + np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)


def scale_exponent(a):
    """Smallest e >= -127 with a <= 448 2^e, for one magnitude a >= 0 (-127 for 0)."""
    if a == 0.0:
        return -127
    m, ex = math.frexp(a)                      # a = m 2^ex, 448 = 0.875 2^9
    return max(ex - 9 if m <= 0.875 else ex - 8, -127)


def quantize(y):
    """float64 [M][K] -> (codes uint8 [M][K], scale bytes uint8 [M][scale_cols(K)])."""
    M, K = y.shape
    codes = np.zeros((M, K), np.uint8)
    scales = np.zeros((M, scale_cols(K)), np.uint8)
    for g in range((K + GROUP - 1) // GROUP):
        part = y[:, g * GROUP:(g + 1) * GROUP]
        for m in range(M):
            if not np.all(np.isfinite(part[m])):
                scales[m, g] = 255
                codes[m, g * GROUP:(g + 1) * GROUP] = 0x7F
                continue
            e = scale_exponent(float(np.max(np.abs(part[m]))))
            scales[m, g] = e + 127
            codes[m, g * GROUP:(g + 1) * GROUP] = encode(np.ldexp(part[m], -e))
    return codes, scales


def dequantize(codes, scales):
    K = codes.shape[1]
    e = np.repeat(scales.astype(np.int64) - 127, GROUP, axis=1)[:, :K]
    v = np.ldexp(VALUES[codes], e)
    v[e == 128] = np.nan
    return v


def product_units(xcodes, xscales, wcodes, wscales, bits=13):
    """2^(E - bits) for one token (xcodes [K]) and weight rows [N][K], per eight consecutive k: E is the
    largest of the eight's sums of both exponents, a subnormal code's being that of the smallest normal
    one.  The 8-bit matrix instruction (bits = 13) cuts each product off there, towards zero.
    float64 [N][K / 8]."""
    def exponents(codes, scales):
        e = np.maximum((codes >> 3 & 15).astype(np.int64), 1) - 7
        return e + np.repeat(scales.astype(np.int64) - 127, GROUP, axis=-1)[..., : codes.shape[-1]]
    e = exponents(wcodes, wscales) + exponents(xcodes, xscales)
    # a product of zero does not count
    e = np.where((wcodes & 0x7F != 0) & (xcodes & 0x7F != 0), e, -1000)
    return np.ldexp(1.0, e.reshape(len(wcodes), -1, 8).max(axis=2) - bits)


def cut_sums(xcodes, xscales, wcodes, wscales, bits=13):
    """Sums over k of one token's products with each weight row, each product cut off towards zero at
    its eight's product_units: float64 [N]."""
    p = dequantize(wcodes, wscales) * dequantize(xcodes[None], xscales[None])
    u = np.repeat(product_units(xcodes, xscales, wcodes, wscales, bits), 8, axis=1)
    return np.sum(np.trunc(p / u) * u, axis=1)


def accumulation_errors(y, target, p):
    """Messages if y [N] is further from target than float32 additions of p [N][K] in any order allow: each
    of K additions is off by half a step of a partial sum (2^-24 of at most sum |p|); and their norm
    over N by what K independent such errors of partial sums of the size of sqrt(sum p^2) add up to."""
    K = p.shape[1]
    err, out = np.abs(y - target), []
    worst = err / (K * 2.0 ** -24 * np.sum(np.abs(p), axis=1) + 1e-300)
    if not np.all(worst <= 1.0):
        out.append(f"row {int(np.nanargmax(worst))}: {np.nanmax(worst):.3g} of the bound")
    norm = np.linalg.norm(err) / (np.sqrt(K) * 2.0 ** -24 * np.linalg.norm(p) + 1e-300)
    if not norm <= 1.0:
        out.append(f"norm: {norm:.3g} of the expected size")
    return out


def rmsnorm(x, residual, gamma, eps):
    """(h, y) in float64 for float64 inputs; residual may be None."""
    h = x if residual is None else x + residual
    return h, h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps) * gamma


def activation(g, act):
    if act == "silu":
        return g / (1.0 + np.exp(-g))
    if act == "gelu":
        from scipy.special import erfc
        return 0.5 * g * erfc(-g / math.sqrt(2.0))
    z = math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)
    return g / (1.0 + np.exp(-2.0 * z))


def gated(xcodes, xscales, wcodes, wscales, act):
    """(g, u, act(g) * u) in float64."""
    y = dequantize(xcodes, xscales) @ dequantize(wcodes, wscales).T
    F = wcodes.shape[0] // 2
    g, u = y[:, :F], y[:, F:]
    return g, u, activation(g, act) * u


def check_codes(codes, scales, y, tau):
    """Errors of codes and scales against float64 values y known to within tau (elementwise):
    each group's scale must be the one of some maximum within tau of y's, and each code the
    rounding of some value within tau of y.  Returns a list of messages."""
    M, K = y.shape
    errors = []
    ng = (K + GROUP - 1) // GROUP
    for g in range(ng):
        sl = slice(g * GROUP, min(K, (g + 1) * GROUP))
        for m in range(M):
            a, t = np.abs(y[m, sl]), tau[m, sl]
            if not np.all(np.isfinite(y[m, sl])):
                if scales[m, g] != 255 or np.any(codes[m, sl] != 0x7F):
                    errors.append(f"row {m} group {g}: not NaN throughout")
                continue
            lo, hi = scale_exponent(max(0.0, float(np.max(a - t)))), scale_exponent(float(np.max(a + t)))
            if not lo + 127 <= int(scales[m, g]) <= hi + 127:
                errors.append(f"row {m} group {g}: scale {scales[m, g]}, expected {lo + 127}..{hi + 127}")
                continue
            e = int(scales[m, g]) - 127
            c = codes[m, sl]
            b = (c & 0x7F).astype(np.int64)
            if np.any(b == 0x7F):
                errors.append(f"row {m} group {g}: NaN code")
                continue
            v, d = np.ldexp(y[m, sl], -e), np.ldexp(t, -e)
            top = np.where(b < 0x7E, MIDPOINTS[np.minimum(b, 0x7D)], 464.0)
            low = np.where(b > 0, MIDPOINTS[np.maximum(b, 1) - 1], -0.0)
            neg = c >= 0x80
            s = np.where(neg, -v, v)                       # the value on the code's side of zero
            bad = (s > top + d) | ((s < low - d) & (b > 0)) | ((b == 0) & (np.abs(v) > top + d))
            if np.any(bad):
                i = int(np.flatnonzero(bad)[0])
                errors.append(f"row {m} col {sl.start + i}: code {c[i]:#x} for {v[i]!r} +- {d[i]!r}")
    if scales.shape[1] > ng and np.any(scales[:, ng:]):
        errors.append("padding bytes of the scales are not zero")
    return errors
