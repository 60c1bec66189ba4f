"""The 8-bit path with exact products (up to 16 tokens, or precise), on the GPU.

Products of 2^16 that cancel in each eight stand beside whole products of at most 9, with scales 2^-1 .. 2 for
each operand: every partial sum is a multiple of 2^-2, below 2^20 in any order within a matrix instruction and
smaller between them, so exact in float32, where 8-bit products keep multiples of 2^3 only.  Every bit equal.
"""

import numpy as np
import pytest
import torch

from oracle import fp8

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _dev(codes, scales):
    return torch.from_numpy(codes).cuda().view(torch.float8_e4m3fn), torch.from_numpy(scales).cuda()


# one shape for each kernel and tile of the linear: up to 64 tokens 16 and 32 weight rows a workgroup, then
# 64 x 64, 128 x 64, 128 x 128, and 256 x 256 (precise: 256 x 128)
SHAPES = [(1, 272), (16, 272), (16, 8208), (17, 272), (32, 4112), (40, 272), (48, 8208), (64, 272), (64, 4112), (100, 272),
          (1000, 1552), (2000, 1552), (3000, 2064)]


def _cancelling(M, N, K, seed):
    """Two products of +-2^16 in each eight that cancel in every output, -3 .. 3 elsewhere, scales 2^-1 .. 2."""
    rng = np.random.default_rng(seed)
    x, w = rng.integers(-3, 4, size=(M, K)).astype(float), rng.integers(-3, 4, size=(N, K)).astype(float)
    for k in range(0, K, 8):
        a, b = k + rng.choice(8, size=2, replace=False)
        x[:, a] = x[:, b] = 256.0 * rng.choice([-1, 1], size=M)
        w[:, a] = 256.0 * rng.choice([-1, 1], size=N)
        w[:, b] = -w[:, a]
    scales = [np.zeros((r, fp8.scale_cols(K)), np.uint8) for r in (M, N)]
    for s in scales:
        s[:, : (K + 127) // 128] = rng.integers(126, 129, size=(len(s), (K + 127) // 128))
    return fp8.encode(x), scales[0], fp8.encode(w), scales[1]


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("K", [16, 144, 656])
def test_cancelling_products_exact(kq, M, N, K):
    xc, xs, wc, ws = _cancelling(M, N, K, M + N)
    bias = torch.from_numpy(np.random.default_rng(1).integers(-9, 10, size=N).astype(np.float64))
    ref = torch.from_numpy(fp8.dequantize(xc, xs) @ fp8.dequantize(wc, ws).T) + bias
    for dtype in (torch.float16, torch.bfloat16):
        y = kq.fp8_linear(*_dev(xc, xs), *_dev(wc, ws), bias=bias.to(dtype).cuda(), dtype=dtype, precise=True)
        assert torch.equal(y.cpu(), ref.to(dtype))
        if M <= 16:
            y = kq.fp8_linear(*_dev(xc, xs), *_dev(wc, ws), bias=bias.to(dtype).cuda(), dtype=dtype)
            assert torch.equal(y.cpu(), ref.to(dtype))


def act_units(g, act):
    """Units 2^-24 of the library's forms: exponential and quotient are good to a few; the tanh form's argument
    comes from five roundings, and an error of it moves the result by |argument| sigmoid(-argument) of it; GELU's
    erfc is moved by g^2 of its argument's error where g < 0."""
    if act == "gelu":
        return 32 + np.where(g < 0, 8 * g * g, 0.0)
    if act == "silu":
        return 16.0
    x = 1.5957691216 * (g + 0.044715 * g ** 3)
    return 16 + 16 * np.abs(x) / (1.0 + np.exp(np.minimum(x, 700.0)))


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M,F,K", [(1, 144, 144), (16, 272, 656), (20, 272, 144), (40, 144, 656), (60, 528, 144), (100, 400, 656),
                                   (700, 5600, 144), (300, 272, 1040)])
def test_gated_cancelling_products(kq, M, F, K, act):
    """Gate and up exact: every code and scale that of the float32 activation."""
    xc, xs, wc, ws = _cancelling(M, 2 * F, K, M + F)
    xs[:, : (K + 127) // 128] -= 6                            # outputs of about unit size, still exact
    g, u, h = fp8.gated(xc, xs, wc, ws, act)
    tau = np.abs(h) * U * (act_units(g, act) + 2) + 2.0 ** -140
    codes, scales = kq.fp8_gated_linear(*_dev(xc, xs), *_dev(wc, ws), act=act, precise=True)
    errors = fp8.check_codes(codes.cpu().view(torch.uint8).numpy(), scales.cpu().numpy(), h, tau)
    assert not errors, errors[:5]
    if M <= 16:
        c, s = kq.fp8_gated_linear(*_dev(xc, xs), *_dev(wc, ws), act=act)
        assert torch.equal(c.view(torch.uint8), codes.view(torch.uint8)) and torch.equal(s, scales)


@pytest.mark.parametrize("M", [20, 100, 400])
def test_precise_nan_and_large_gates(kq, M):
    """A NaN group makes NaN exactly the outputs that use it; gates far out on both sides stay finite."""
    N, K = 288, 400
    rng = np.random.default_rng(M)
    xc, wc = fp8.encode(rng.integers(-3, 4, size=(M, K)).astype(float)), fp8.encode(rng.integers(-3, 4, size=(N, K)).astype(float))
    xs, ws = np.zeros((M, 4), np.uint8), np.zeros((N, 4), np.uint8)
    xs[:], ws[:] = 127, 127
    xc[M - 1, 256:384], xs[M - 1, 2] = 0x7F, 255
    wc[33, 384:], ws[33, 3] = 0x7F, 255
    y = kq.fp8_linear(*_dev(xc, xs), *_dev(wc, ws), dtype=torch.bfloat16, precise=True).cpu()
    ref = torch.from_numpy(fp8.dequantize(xc, xs) @ fp8.dequantize(wc, ws).T).to(torch.bfloat16)
    assert torch.equal(torch.isnan(y), torch.isnan(ref))
    assert torch.equal(torch.nan_to_num(y), torch.nan_to_num(ref))
    wc[33, 384:], ws[33, 3] = 0, 127
    xs[: M - 1, :] += 6
    for act in ("silu", "gelu", "gelu_tanh"):
        codes, scales = kq.fp8_gated_linear(*_dev(xc, xs), *_dev(wc, ws), act=act, precise=True)
        codes, scales = codes.cpu().view(torch.uint8).numpy(), scales.cpu().numpy()
        with np.errstate(over="ignore", under="ignore"):
            g, u, h = fp8.gated(xc[:-1], xs[:-1], wc, ws, act)
        tau = np.abs(h) * U * (act_units(g, act) + 2) + np.abs(u) * 2.0 ** -100
        assert not fp8.check_codes(codes[:-1], scales[:-1], h, tau), act
        assert np.all(codes[-1] == 0x7F) and np.all(scales[-1, :2] == 255)


@pytest.mark.parametrize("M", [1, 40, 300])
def test_precise_captured_and_replayed(kq, M):
    """A captured gated pair and down-projection of exact products, replayed on new inputs with eager work and waits
    between, gives the eager bytes each time."""
    F, D = 528, 272
    weights = [_dev(*fp8.quantize(np.random.default_rng(s).normal(size=n) / 16)) for s, n in ((1, (2 * F, D)), (2, (D, F)))]
    x = torch.empty(M, D, dtype=torch.bfloat16, device="cuda")

    def block():
        codes, scales = kq.fp8_gated_linear(*kq.quantize_fp8(x), *weights[0], act="gelu", precise=True)
        return codes, scales, kq.fp8_linear(codes, scales, *weights[1], dtype=torch.bfloat16, precise=True)
    x.normal_()
    block()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block()
    for k in range(3):
        x.copy_(torch.randn(M, D, generator=torch.Generator().manual_seed(k)).cuda())
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, block()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), k
        torch.cuda.synchronize()
