"""kq.h's promise that the binding relies on: kq_attention needs no workspace up to 704 keys."""

import random

import w4a4_post_quantization_amd as kq


def test_none_up_to_704_keys():
    rng = random.Random(0)
    need = kq.load().kq_attention_workspace_bytes
    some = 0
    for _ in range(20000):
        Hkv = rng.choice([1, 2, 3, 4, 8, 16, 64])
        Hq, D = Hkv * rng.choice([1, 2, 5, 16]), rng.choice([8, 64, 72, 96, 128])
        B, T, packed = rng.choice([1, 1, 2, 30, 300]), int(10 ** rng.uniform(0, 4)), rng.randrange(2)
        assert need(B, T, rng.randint(1, 704), packed, Hq, Hkv, D) == 0
        some += need(B, T, rng.randint(705, 20000), packed, Hq, Hkv, D) > 0
    assert some > 1000
