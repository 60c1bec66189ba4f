"""Refusals of the 8-bit path's flag for exact products."""

import ctypes

import w4a4_post_quantization_amd as kq

P = ctypes.c_void_p(0x100000)          # never dereferenced: the calls are refused first
PRECISE, UNSUPPORTED, SHAPE = 0x100, 4, 2


def test_precise_flag_refusals():
    lib = kq.load()

    def linear(dt, M=4):
        return lib.kq_fp8_linear(dt, P, P, M, 64, P, P, 32, None, P, None)

    def gated(act, M=4):
        return lib.kq_fp8_gated_linear(act, P, P, M, 64, P, P, 32, P, P, P, 1 << 40, None)
    for f in (linear, gated):
        for bad in (3 | PRECISE, 0x200, 0x200 | PRECISE, -1):
            assert f(bad) == UNSUPPORTED
        for ok in (0, 1):
            assert f(ok | PRECISE, M=0) == SHAPE            # the flag is taken, the next check refuses
