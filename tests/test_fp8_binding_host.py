"""Refusals of the 8-bit binding that need no GPU: what would be dropped silently, and arguments that are no tensors."""

import pytest
import torch

import w4a4_post_quantization_amd as kq

X = torch.zeros(4, 64, dtype=torch.float16)


def test_residual_out_without_a_residual():
    """It would never be written."""
    with pytest.raises(ValueError, match="residual_out"):
        kq.rmsnorm_quantize_fp8(X, X[0], residual_out=torch.zeros_like(X))
