"""GPU: a NaN among what a row sees reaches its output and its lse, wherever it lies in the division of
the work: alone in a wave's steps, in every key of a range, in the query itself. Compared with a
64-bit evaluation (tests/attn_ref.py), lse included; what does not see the NaN stays exact."""
import math

import pytest
import torch

import attn_ref
import gated_deltanet_linear_prefill_amd as gdn
from test_gpu_attn_decode import dense, fill, queries
from test_gpu_attn_prefill import compare as compare_prefill
from test_gpu_attn_prefill import make, offsets, run
from test_gpu_kv_cache import BF, DEV, F8, F32, Cache, ints

pytestmark = pytest.mark.gpu

STORES = [(BF, BF), (BF, F8), (F32, F32), (F32, F8)]


def spoil(cache, name, s, pos, head, el):
    """NaN in one element of a row that is there."""
    page, row = cache.place(s, pos)
    pool = getattr(cache, name)
    if cache.store == F8:
        pool.view(torch.uint8)[page, head, row, el] = 0x7f
    else:
        pool[page, head, row, el] = math.nan


def check_decode(cache, q, lens, out, lse):
    g, d = q.shape[1] // cache.h, q.shape[2]
    for s, length in enumerate(lens):
        k, v, there = dense(cache, s, length)
        for h in range(q.shape[1]):
            ref = attn_ref.attend(q[s:s + 1, h], k[:, h // g], v[:, h // g], d ** -0.5, there[None])
            what = f"sequence {s} of {length}, head {h}"
            attn_ref.check(out[s:s + 1, h], lse[s:s + 1, h], *ref, what=what)
            assert torch.equal(torch.isnan(lse[s:s + 1, h]).cpu(), torch.isnan(ref[1])), what + ": NaN in lse"


def decode(cache, q, lens):
    lse = torch.full(q.shape[:2], 5.0, device=DEV)
    out = gdn.gdn_attn_decode(q.to(DEV), *cache.args(), ints(lens), lse=lse, **cache.scales())
    check_decode(cache, q, lens, out, lse)
    return out, lse


@pytest.mark.parametrize("dtype,store", STORES)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode_nan_in_a_query(dtype, store, d):
    lens = [1, 33, 200, 3000]
    cache = Cache(lens, 16, 2, d, store)
    fill(cache, d, nan_behind=lens)
    q = queries(4, 6, d, dtype)
    q[:, 1, 3] = math.nan
    q[2, 5, d - 1] = math.nan
    out, lse = decode(cache, q, lens)
    bad = torch.zeros(4, 6, dtype=torch.bool)
    bad[:, 1] = bad[2, 5] = True
    assert torch.equal(torch.isnan(lse).cpu(), bad)
    assert torch.equal(torch.isnan(out).cpu(), bad[..., None].expand(out.shape))


# The last position is alone in its wave's steps of 16 or 32 positions, or in its workgroup's range.
LAST = [1, 16, 17, 33, 49, 65, 97, 129, 257, 513, 1025, 3073]


@pytest.mark.parametrize("dtype,store", STORES)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode_nan_in_the_newest_key(dtype, store, d):
    cache = Cache(LAST, 16, 2, d, store)
    fill(cache, 1 + d, nan_behind=LAST)
    for s, length in enumerate(LAST):
        spoil(cache, "k", s, length - 1, 0, length % d)
    out, lse = decode(cache, queries(len(LAST), 4, d, dtype), LAST)
    assert bool(torch.isnan(out[:, :2]).all()) and not bool(torch.isnan(out[:, 2:]).any())
    assert bool(torch.isnan(lse[:, :2]).all()) and not bool(torch.isnan(lse[:, 2:]).any())


@pytest.mark.parametrize("dtype,store", STORES)
def test_decode_nan_in_every_key_of_a_range(dtype, store):
    """One sequence whose cache is divided: NaN in all keys of the middle third, of the first position only,
    and of every key."""
    d, length = 128, 3000
    for at in (range(1000, 2000), range(1), range(length)):
        cache = Cache([length], 64, 1, d, store)
        fill(cache, 9)
        assert gdn.gdn_attn_decode_workspace_bytes(1, cache.page_table.shape[1], 64, 2, 1, d, length, store) > 0
        for pos in at:
            spoil(cache, "k", 0, pos, 0, 7)
        out, lse = decode(cache, queries(1, 2, d, dtype), [length])
        assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())


@pytest.mark.parametrize("dtype,store", STORES)
def test_decode_nan_in_a_value(dtype, store):
    """A NaN in V reaches its own element only, and not lse."""
    lens = [1, 17, 33, 2500]
    cache = Cache(lens, 16, 1, 64, store)
    fill(cache, 11)
    for s, length in enumerate(lens):
        spoil(cache, "v", s, length - 1, 0, 5)
    out, lse = decode(cache, queries(4, 2, 64, dtype), lens)
    assert bool(torch.isnan(out[..., 5]).all()) and int(torch.isnan(out).sum()) == 8
    assert bool(torch.isfinite(lse).all())


# few rows over many keys (divided), short prompts, many tiles
PREFILLS = [([5], [4000], 4, 2, 128), ([3, 1, 40], [3, 700, 41], 4, 2, 256), ([300], [300], 2, 1, 64), ([1100], [1100], 2, 1, 128)]


@pytest.mark.parametrize("lq,lk,hq,hk,d", PREFILLS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_nan_in_queries_and_keys(lq, lk, hq, hk, d, dtype):
    q, k, v = make(lq, lk, hq, hk, d, dtype, seed=d)
    cq, ck = offsets(lq), offsets(lk)
    row = cq[-1] - 1
    q[0, 0, 1] = math.nan       # one head of the first row
    k[ck[-1] - 1, hk - 1, 2] = math.nan  # seen by the last row alone, in the last KV head
    out, lse = run(q, k, v, lq, lk)
    compare_prefill(q, k, v, lq, lk, True, d ** -0.5, out, lse)
    bad = torch.zeros(q.shape[:2], dtype=torch.bool)
    bad[0, 0] = True
    bad[row, hq - hq // hk:] = True
    assert torch.equal(torch.isnan(lse).cpu(), bad)
    assert torch.equal(torch.isnan(out).cpu(), bad[..., None].expand(out.shape))
