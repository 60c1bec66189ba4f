"""The 8-bit products to each side of the rules that choose between weight rows and tiles."""

import numpy as np
import pytest
import torch

from oracle import fp8

pytestmark = pytest.mark.gpu


def _whole(rows, K, seed):
    """Codes of whole numbers -3 .. 3 with scales 2^-1 .. 2 and their float64 values, on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ng = (K + 127) // 128
    codes = torch.randint(-3, 4, (rows, K), device="cuda", generator=g).float().to(torch.float8_e4m3fn)
    scales = torch.zeros(rows, fp8.scale_cols(K), dtype=torch.uint8, device="cuda")
    scales[:, :ng] = torch.randint(126, 129, (rows, ng), device="cuda", generator=g, dtype=torch.uint8)
    unit = torch.exp2(scales[:, :ng].double() - 127).repeat_interleave(128, 1)[:, :K]
    return codes, scales, codes.double() * unit


def test_gated_workspace_follows_the_compute_units(kq):
    """Rows (and their float32 outputs) while the workgroups of 16 columns all run at once."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    for M, per in ((33, 3), (48, 3), (49, 2), (64, 2)):
        F = 16 * per * cus
        assert kq.fp8_gated_linear_workspace_bytes(M, F, 128) == 4 * M * F
        assert kq.fp8_gated_linear_workspace_bytes(M, F + 16, 128) == 0
    assert kq.fp8_gated_linear_workspace_bytes(32, 1 << 19, 128) == 4 * 32 << 19
    assert kq.fp8_gated_linear_workspace_bytes(65, 16, 128) == 0


@pytest.mark.parametrize("M", [33, 48, 49, 64])
def test_gated_to_each_side(kq, M):
    """The same columns give the same bytes' values with one workgroup more than the rule allows."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    F, K = 16 * (3 if M <= 48 else 2) * cus, 144
    x, xs, xv = _whole(M, K, M)
    xs[:, :2] -= 6
    w, ws, wv = _whole(2 * (F + 16), K, F)
    h = []
    for cols in (F, F + 16):
        rows = torch.cat([torch.arange(cols), F + 16 + torch.arange(cols)]).cuda()
        codes, scales = kq.fp8_gated_linear(x, xs, w.view(torch.uint8)[rows].view(torch.float8_e4m3fn), ws[rows])
        h.append(codes[:, :F].double() * torch.exp2(scales[:, : F // 128].double() - 127).repeat_interleave(128, 1))
    y = xv / 64 @ wv.t()
    exact = y[:, :F] * torch.sigmoid(y[:, :F]) * y[:, F + 16:2 * F + 16]
    top = exact.abs().view(M, -1, 128).amax(2).repeat_interleave(128, 1)
    # half a step of E4M3 (2^-4 of the value; below its normal numbers 2^-10 of a unit of at most 2^-7.8 of the
    # group's largest), and 1e-5 for the float32 activation
    for v in h:
        assert bool(((v - exact).abs() <= torch.maximum(exact.abs() * 2.0 ** -4, top * 2.0 ** -17) + 1e-5 * exact.abs()).all())


@pytest.mark.parametrize("M", [32, 33, 48, 49, 64])
@pytest.mark.parametrize("K", [144, 656])
@pytest.mark.parametrize("precise", [False, True])
def test_linear_to_each_side(kq, M, K, precise):
    """Every bit, with as many workgroups of 32 weight rows as the rule allows and one more."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    N = 32 * (3 if M <= 48 else 2) * cus
    x, xs, xv = _whole(M, K, M)
    w, ws, wv = _whole(N + 16, K, N)
    ref = (xv @ wv.t()).to(torch.float16)                    # sums exact in float32
    for n in (N, N + 16):
        y = kq.fp8_linear(x, xs, w[:n], ws[:n], precise=precise)
        assert torch.equal(y, ref[:, :n])
