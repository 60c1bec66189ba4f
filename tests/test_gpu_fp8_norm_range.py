"""The norm of rows near the ends of float32: sums of squares and factors that float32 cannot hold."""

import numpy as np
import pytest
import torch

from oracle import fp8

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("K", [16, 640, 4096, 6000, 16384])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_rows_of_any_size(kq, K, eps):
    """Each row its own size, from subnormal to the largest bf16; the tolerance is that of rows of ordinary size
    (64 u of y: one more rounding, the factor's first part; a power of two moves nothing), and for values whose
    bf16 is subnormal nothing more, for they are float32 values too."""
    sizes = [1e-39, 1e-30, 1e-22, 3e-19, 1e-16, 1.0, 1e15, 5e17, 3e18, 1e19, 1e25, 1e33, 5e37]
    rng = np.random.default_rng(K)
    x = torch.from_numpy(np.array(sizes)[:, None] * rng.normal(size=(len(sizes), K)).clip(-3, 3)).to(torch.bfloat16)
    x[:, 0] = torch.tensor(sizes).to(torch.bfloat16)         # no row is all zeros
    x[-1, 1] = torch.finfo(torch.bfloat16).max
    gamma = torch.from_numpy(1.0 + 0.3 * rng.normal(size=K)).to(torch.bfloat16)
    codes, scales, _ = kq.rmsnorm_quantize_fp8(x.cuda(), gamma.cuda(), eps=eps)
    _, y = fp8.rmsnorm(x.double().numpy(), None, gamma.double().numpy(), float(np.float32(eps)))
    errors = fp8.check_codes(codes.cpu().view(torch.uint8).numpy(), scales.cpu().numpy(), y, 64 * U * np.abs(y) + 2.0 ** -149)
    assert not errors, errors[:5]


def test_residual_of_large_rows_is_kept(kq):
    """residual_out is the sum itself, not its scaled form; ordinary rows beside large ones keep their bytes."""
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.normal(size=(6, 512))).to(torch.bfloat16)
    r = torch.from_numpy(rng.normal(size=(6, 512))).to(torch.bfloat16)
    gamma = torch.ones(512, dtype=torch.bfloat16)
    c0, s0, h0 = kq.rmsnorm_quantize_fp8(x.cuda(), gamma.cuda(), residual=r.cuda())
    x[2:4] *= 1e25
    r[2:4] *= 1e25
    c, s, h = kq.rmsnorm_quantize_fp8(x.cuda(), gamma.cuda(), residual=r.cuda())
    assert torch.equal(h.cpu(), (x.float() + r.float()).to(torch.bfloat16))
    keep = [0, 1, 4, 5]
    assert torch.equal(c.view(torch.uint8)[keep], c0.view(torch.uint8)[keep]) and torch.equal(s[keep], s0[keep])
    _, y = fp8.rmsnorm((x.float() + r.float()).double().numpy(), None, np.ones(512), 1e-6)
    assert not fp8.check_codes(c.cpu().view(torch.uint8).numpy(), s.cpu().numpy(), y, 64 * U * np.abs(y))
    # a row of zeros without eps has no direction
    z = torch.zeros(2, 512, dtype=torch.bfloat16, device="cuda")
    c, s, _ = kq.rmsnorm_quantize_fp8(z, gamma.cuda(), eps=0.0)
    assert bool((c.view(torch.uint8) == 0x7F).all()) and bool((s == 255).all())
