"""CPU: the workspace of gdn_attn_extend, for batches that mix many short sequences with a long piece above all."""
import random

import pytest
import torch

import gated_deltanet_linear_prefill_amd as gdn

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def serves_every_call(d):
    """The size that include/gdn.h gives: at most 10240 parts of 32 (d = 256) or 64 rows for sequences of few rows, and 1024
    of 256 rows for those of many."""
    return (10240 * (32 if d == 256 else 64) + 262144) * (4 * d + 16)


# one piece of a prompt among sequences that bring a token each: n, tokens, h_q, h_kv, d, max_q, max_len, dtype, store
MIXED = [
    (512, 732, 8, 8, 256, 128, 131072, BF, F8), (1000, 1100, 1, 1, 256, 101, 131072, BF, BF), (256, 768, 8, 1, 256, 513, 131072, BF, F8),
    (256, 767, 32, 8, 128, 512, 131072, BF, BF), (193, 3107, 8, 8, 256, 3107, 84046, BF, F8), (512, 800, 16, 2, 256, 289, 65536, F32, F32),
    (100, 600, 16, 2, 256, 501, 131072, F32, F8), (2000, 2500, 32, 8, 128, 501, 131072, BF, F8), (65, 200, 16, 16, 64, 136, 131072, BF, BF),
    (1 << 22, 800, 8, 8, 256, 129, 131072, BF, F8),  # the grid of a join would pass 2^31 workgroups
]


@pytest.mark.parametrize("n,total,hq,hk,d,max_q,max_len,dtype,store", MIXED)
def test_a_long_piece_among_many_tokens(n, total, hq, hk, d, max_q, max_len, dtype, store):
    need = gdn.gdn_attn_extend_workspace_bytes(n, max_len // 16, 16, total, hq, hk, d, max_q=max_q, max_len=max_len, dtype=dtype, store=store)
    assert need <= serves_every_call(d)


@pytest.mark.parametrize("most_sequences", [6, 11, 18])
def test_one_buffer_serves_every_call(most_sequences):
    rng = random.Random(most_sequences)
    size = lambda top: int(2 ** rng.uniform(0, top))
    seen = 0
    for _ in range(30000):
        hk, g, n, d = rng.choice([1, 2, 3, 8, 16]), rng.choice([1, 2, 3, 8, 16, 20, 64]), size(most_sequences), rng.choice([64, 128, 256])
        total, dtype = size(16), rng.choice([BF, BF, F32])
        need = gdn.gdn_attn_extend_workspace_bytes(
            n, size(18), rng.choice([16, 64, 1024]), total, hk * g, hk, d, max_q=rng.choice([1, size(10), total]), max_len=size(22),
            window=rng.choice([0, 0, size(16)]), sinks=size(8), dtype=dtype, store=rng.choice([dtype, F8]))
        assert 0 <= need <= serves_every_call(d)
        seen += need > 0
    assert seen > 3000
