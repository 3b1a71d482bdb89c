"""GPU: prefill attention with a few more tiles than the chip takes at a time (257 to 511 tiles of 256
rows), where the choice between the workgroup shapes changes. Sampled rows are compared."""
import random

import pytest

from test_gpu_attn_prefill import make, run
from test_gpu_attn_shapes import sampled
from test_gpu_kv_cache import BF

pytestmark = pytest.mark.gpu


# (tokens, keys, heads, KV heads, d): tiles from 257 to 511, the edges among them
SIZES = [(4112, 4112, 16, 2, 256), (4352, 4352, 16, 2, 256), (5120, 5120, 16, 2, 256), (6144, 6500, 16, 2, 256),
         (8180, 8180, 16, 2, 256), (4100, 4100, 16, 16, 128), (2900, 3100, 32, 8, 64), (4111, 4111, 16, 1, 256)]


@pytest.mark.parametrize("lq,lk,hq,hk,d", SIZES)
def test_sampled_rows(lq, lk, hq, hk, d):
    q, k, v = make([lq], [lk], hq, hk, d, BF, seed=lq)
    out, lse = run(q, k, v, [lq], [lk])
    r = random.Random(lq)
    sampled(q, k, v, lq, lk, out, lse, [0, 1, 31, 127, 128, 255, 256, lq // 2, lq - 129, lq - 2, lq - 1] + [r.randrange(lq) for _ in range(12)])
