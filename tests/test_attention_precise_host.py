"""The flag for precise weights changes no refusal of kq_attention's."""

import ctypes

import pytest

import w4a4_post_quantization_amd as kq

P = ctypes.c_void_p(0x100000)          # never dereferenced: the call is refused first
PRECISE = 0x100
SHAPE, UNSUPPORTED, WORKSPACE = 2, 4, 7


@pytest.mark.parametrize("dtype,T,Tk,status", [(PRECISE, 0, 5, SHAPE), (1 | PRECISE, 5, 0, SHAPE), (2 | PRECISE, 5, 5, UNSUPPORTED),
                                               (2 * PRECISE, 5, 5, UNSUPPORTED), (1 | PRECISE, 10, 5000, WORKSPACE)])
def test_refusals(dtype, T, Tk, status):
    assert kq.load().kq_attention(dtype, P, 512, 128, P, 256, 128, P, 256, 128, None, None, 1, T, Tk, 4, 2, 128, 1, 0.1, P, None,
                                  None, None, 0, None) == status
