"""Refusals of the 8-bit binding behind its checks of the operands."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_arguments_that_are_no_tensors(kq):
    x = kq.quantize_fp8(torch.zeros(4, 64, dtype=torch.float16, device="cuda"))
    w = kq.quantize_fp8(torch.zeros(32, 64, dtype=torch.float16, device="cuda"))
    for bad in ("Y", 7, [1.0]):
        for name in ("bias", "Y"):
            with pytest.raises(ValueError):
                kq.fp8_linear(*x, *w, **{name: bad})
            with pytest.raises(ValueError):
                kq.fp8_linear(*x, *w, dtype=torch.float16, **{name: bad})
        for name in ("codes", "scales", "workspace"):
            with pytest.raises(ValueError):
                kq.fp8_gated_linear(*x, *w, **{name: bad})
