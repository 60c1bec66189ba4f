"""Shared by the attention tests: inputs, the oracle's tolerances, comparison."""

import numpy as np
import torch

from oracle import fp8

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
HALF = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}             # half a step, relative
# A prompt's weight is rounded to the 16-bit type of the second product; fp16 ones are held at 2^6 of the largest or more,
# so what falls below fp16's smallest step of 2^-24 is at most 2^-31 of the largest weight.  The paged cache's weights are
# sums of such numbers and allow less: paged_pairs.WEIGHT.
WEIGHT = {("fp16", "fp16"): (2.0 ** -11, 2.0 ** -31), ("bf16", "bf16"): (2.0 ** -8, 0.0),
          ("fp16", "fp8"): (2.0 ** -16, 0.0), ("bf16", "fp8"): (2.0 ** -8, 0.0)}


def dbl(t):
    return t.detach().cpu().double().numpy()


def raw(t):
    return t.detach().cpu().contiguous().view(torch.uint8).numpy()


def heads(shape, dtype, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    x = spread * rng.normal(size=shape) + 0.3 * rng.normal(size=shape[-2:])
    return torch.from_numpy(x).to(DT[dtype]).cuda()


def cumulative(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)


def on_gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check(y, o, tau, dtype, label=""):
    """y (16-bit) against o float64: tau, and half a step of the type (or of its smallest one)."""
    y = dbl(y)
    assert np.array_equal(np.isnan(y), np.isnan(o)), label
    inf = np.isinf(o)
    assert np.array_equal(y[inf], o[inf]), label
    ok = np.isfinite(o)
    err = np.abs(y[ok] - o[ok])
    bound = tau[ok] + HALF[dtype] * (np.abs(o[ok]) + tau[ok]) + (2.0 ** -25 if dtype == "fp16" else 2.0 ** -134)
    worst = np.max(err / bound) if err.size else 0.0
    assert worst <= 1.0, f"{label}: {worst:.3g} of the bound"


def check_codes(codes, scales, o, tau):
    """Codes and scales of rows [n][H][128]; the padding's bytes are zero."""
    n, H, _ = o.shape
    bad = fp8.check_codes(raw(codes).reshape(n, -1), raw(scales).reshape(n, -1), o.reshape(n, -1), tau.reshape(n, -1))
    assert not bad, bad[:3]


def quantized(x):
    """float64 rows [...][D] -> (codes, scale bytes) of each row as a group."""
    rows = x.reshape(-1, x.shape[-1])
    codes, scales = fp8.quantize(rows)
    return codes.reshape(x.shape), scales[:, 0].reshape(x.shape[:-1])


def widened(codes, scales):
    v = fp8.VALUES[codes]
    return np.ldexp(v, scales.astype(np.int64)[..., None] - 127)


class Cache:
    """A cache with pages in random order, garbage (NaN) wherever no token is."""

    def __init__(self, lengths, Hkv, D, page, dtype, cache, seed, spare=2, width=None, hole=False):
        rng = np.random.default_rng(seed)
        need = [-(-max(n, 0) // page) for n in lengths]
        self.page, self.pages = page, sum(need) + spare
        self.width = max([1, *need]) if width is None else width
        order = rng.permutation(self.pages).astype(np.int32)
        self.table = np.full((len(lengths), self.width), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.lengths = np.array(lengths, np.int32)
        shape = (self.pages, Hkv, page, D)
        k = rng.normal(size=shape) + 0.3 * rng.normal(size=(1, Hkv, 1, D))
        v = rng.normal(size=shape) * np.exp(0.5 * rng.normal(size=(*shape[:3], 1)))
        used = np.zeros((self.pages, page), bool)
        for b, n in enumerate(lengths):
            for j in range(max(n, 0)):
                used[self.table[b, j // page], j % page] = True
        self.ks = self.vs = None
        if cache == "fp8":
            (ck, sk), (cv, sv) = quantized(k), quantized(v)
            self.k64, self.v64 = widened(ck, sk), widened(cv, sv)
            for c, s in ((ck, sk), (cv, sv)):
                c[:] = np.where(used[:, None, :, None], c, 0x7F)
                s[:] = np.where(used[:, None, :], s, 255)
            self.k, self.v = (on_gpu(c).view(torch.float8_e4m3fn) for c in (ck, cv))
            self.ks, self.vs = on_gpu(sk), on_gpu(sv)
        else:
            k, v = (np.where(used[:, None, :, None], t, np.nan) for t in (k, v))
            self.k, self.v = (torch.from_numpy(t).to(DT[dtype]).cuda() for t in (k, v))
            self.k64, self.v64 = dbl(self.k), dbl(self.v)
        if hole:                                              # a page that is not there, one beyond the cache
            b = int(np.argmax(need))
            self.table[b, need[b] // 2] = -7
            self.table[b, 0] = self.pages

    def args(self):
        return self.k, self.v, on_gpu(self.table), on_gpu(self.lengths)

    def scales(self):
        return dict(kscales=self.ks, vscales=self.vs)
