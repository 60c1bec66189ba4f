"""Tensors without elements are refused by the attention's binding, by name."""

import pytest
import torch

import w4a4_post_quantization_amd as kq

H = torch.zeros(4, 2, 64, dtype=torch.float16)


@pytest.mark.parametrize("shape", [(0, 2, 64), (4, 0, 64), (4, 2, 0)])
def test_empty(shape):
    E = torch.zeros(shape, dtype=torch.float16)
    for call in (lambda: kq.attention(E, H, H), lambda: kq.cache_append(E, H, H, H, H, H),
                 lambda: kq.paged_attention(E, H, H, H, H)):
        with pytest.raises(ValueError, match="at least one"):
            call()


def test_no_keys():
    with pytest.raises(ValueError, match="K must hold at least one"):
        kq.attention(H, H[:0], H[:0], torch.tensor([0, 4], dtype=torch.int32), torch.tensor([0, 0], dtype=torch.int32))
