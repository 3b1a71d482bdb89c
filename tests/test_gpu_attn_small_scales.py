"""GPU: scales that are zero or close to it, with scores that large queries and keys make: every finite scale
is used as it is."""
import pytest
import torch

import attn_ref
import gated_deltanet_linear_prefill_amd as gdn
from test_gpu_attn_decode import compare as compare_decode
from test_gpu_attn_decode import fill, queries
from test_gpu_attn_prefill import compare, make, run
from test_gpu_kv_cache import BF, DEV, F32, Cache, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [0.0, -0.0, 2e-38, -2e-38, 1e-40])
@pytest.mark.parametrize("lq,lk", [([150], [150]), ([4], [3000])])
def test_prefill(dtype, scale, lq, lk):
    # scores before the scale are up to about 1e38
    q, k, v = make(lq, lk, 2, 1, 64, dtype, spread=2.0 ** 61)
    k = k * 2.0 ** 60
    out, lse = run(q, k, v, lq, lk, True, scale)
    assert bool(torch.isfinite(out).all())
    compare(q, k, v, lq, lk, True, scale, out, lse, f"scale {scale}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [0.0, 1e-39, -1e-39])
@pytest.mark.parametrize("lq,lk", [([300], [300]), ([1200], [1200]), ([4], [3000])])
def test_prefill_scores_of_both_ends(dtype, scale, lq, lk):
    """Scores before the scale near the largest float, negative ones first: their difference is past it."""
    q, k, v = make(lq, lk, 2, 1, 64, dtype)
    q.zero_()
    k.zero_()
    q[..., 5] = 2.0 ** 63
    k[:, :, 5] = 1.25 * 2.0 ** 64
    k[:lk[0] // 2] *= -1
    out, lse = run(q, k, v, lq, lk, True, scale)
    compare(q, k, v, lq, lk, True, scale, out, lse, f"scale {scale}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [0.0, 2e-38, -2e-38, 1e-40])
def test_decode(dtype, scale):
    lens = [150, 3000]
    cache = Cache(lens, 16, 1, 64, dtype)
    fill(cache, 3)
    cache.k *= 2.0 ** 60
    q = queries(2, 2, 64, dtype) * 2.0 ** 60
    lse = torch.zeros(2, 2, device=DEV)
    out = gdn.gdn_attn_decode(q.to(DEV), *cache.args(), ints(lens), scale=scale, lse=lse)
    compare_decode(cache, q, lens, out, lse, scale)
