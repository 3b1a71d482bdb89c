"""GPU: attention at seeded random shapes, and at sizes that reach every division of the work
(tests/attn_ref.py has the 64-bit evaluation and the bounds). Large cases compare sampled rows."""
import math
import random

import pytest
import torch

import attn_ref
import gated_deltanet_linear_prefill_amd as gdn
from test_gpu_attn_decode import compare as compare_decode
from test_gpu_attn_decode import fill, queries
from test_gpu_attn_prefill import compare, ints, make, offsets, run
from test_gpu_kv_cache import BF, DEV, F8, F32, Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", range(24))
def test_random_prefills(seed):
    r = random.Random(seed)
    dtype, d = r.choice([BF, BF, F32]), r.choice([64, 128, 256])
    hk, g, n = r.choice([1, 2, 3]), r.choice([1, 2, 3, 5, 8]), r.randint(1, 6)
    lq = [r.choice([0, 1, r.randint(1, 64), r.randint(1, 700)]) for _ in range(n)]
    lk = [max(0, x + r.choice([0, 0, 1, r.randint(0, 300), -r.randint(0, 40)])) for x in lq]
    causal, scale = r.random() < 0.7, r.choice([None, 0.05, 0.5])
    q, k, v = make(lq, lk, hk * g, hk, d, dtype, seed=seed)
    out, lse = run(q, k, v, lq, lk, causal, scale)
    compare(q, k, v, lq, lk, causal, d ** -0.5 if scale is None else scale, out, lse, f"{lq} {lk}")


@pytest.mark.parametrize("seed", range(24))
def test_random_decodes(seed):
    r = random.Random(1000 + seed)
    dtype, d = r.choice([BF, BF, F32]), r.choice([64, 128, 256])
    store = r.choice([dtype, F8])
    hk, g, n = r.choice([1, 2, 3]), r.choice([1, 2, 4, 8, 17]), r.randint(1, 5)
    lens = [r.choice([0, 1, r.randint(1, 64), r.randint(1, 1500)]) for _ in range(n)]
    cache = Cache(lens, r.choice([16, 32, 128]), hk, d, store, seed=seed)
    fill(cache, seed, nan_behind=lens)
    q = queries(n, hk * g, d, dtype, seed)
    lse = torch.zeros(n, hk * g, device=DEV)
    out = gdn.gdn_attn_decode(q.to(DEV), *cache.args(), ints(lens), max_len=max(lens) + r.choice([0, 3]), lse=lse,
                              **cache.scales())
    compare_decode(cache, q, lens, out, lse, d ** -0.5)


def sampled(q, k, v, lq, lk, out, lse, rows, what=""):
    """Compare some rows of one causal sequence."""
    g, d = q.shape[1] // k.shape[1], q.shape[2]
    at = torch.tensor(rows)
    allowed = attn_ref.causal_mask(lq, lk, True)[at]
    for h in range(q.shape[1]):
        kk, vv = k[:, h // g].clone(), v[:, h // g].clone()
        unseen = ~allowed.any(0)
        kk[unseen], vv[unseen] = 0, 0
        ref = attn_ref.attend(q[at, h], kk, vv, d ** -0.5, allowed)
        attn_ref.check(out[at, h], None if lse is None else lse[at, h], *ref, what=f"{what} head {h}")


# (queries, keys, heads, KV heads, d): 256 tiles of 256 rows or fewer with many keys; more tiles with
# 8192 keys or more and d = 256; more tiles otherwise
LARGE = [(1300, 1300, 4, 2, 128, BF), (1100, 2100, 2, 1, 64, BF), (1030, 1030, 4, 1, 256, BF), (1200, 1200, 2, 2, 64, F32),
         (1060, 1060, 2, 1, 128, F32), (1040, 1040, 1, 1, 256, F32), (4200, 8300, 16, 2, 256, BF), (2100, 2100, 32, 8, 128, BF),
         (9000, 9000, 8, 8, 64, BF)]


@pytest.mark.parametrize("with_lse", [False, True])
@pytest.mark.parametrize("lq,lk,hq,hk,d,dtype", LARGE)
def test_large_prefills(lq, lk, hq, hk, d, dtype, with_lse):
    q, k, v = make([lq], [lk], hq, hk, d, dtype, seed=d + lq)
    out, lse = run(q, k, v, [lq], [lk], True, None, with_lse)
    r = random.Random(lq)
    rows = [0, 1, 31, 32, 63, 127, 128, lq - 2, lq - 1] + [r.randrange(lq) for _ in range(20)]
    sampled(q, k, v, lq, lk, out, lse, rows)
    if with_lse:  # asking for lse does not change the output
        assert torch.equal(out, run(q, k, v, [lq], [lk], True, None, False)[0])


@pytest.mark.parametrize("lq,lk,hq,hk,d,dtype", [LARGE[0], LARGE[2], LARGE[3], LARGE[6], LARGE[7]])
@pytest.mark.parametrize("bad", [math.nan, -math.inf])
def test_bad_values_behind_what_a_row_sees(lq, lk, hq, hk, d, dtype, bad):
    q, k, v = make([lq], [lk], hq, hk, d, dtype, seed=1)
    first = lq - 90  # rows before it see none of these
    k[lk - 50:], v[first + lk - lq:] = bad, bad
    out, _ = run(q, k, v, [lq], [lk], True, None, False)
    sampled(q, k, v, lq, lk, out, None, [0, 40, first // 2, first - 33, first - 2, first - 1])
    assert not bool(torch.isfinite(out[first:].float()).any())


# 256 tiles of 256 rows or fewer with many keys, and enough of them that keys are not divided
BUSY = [(2000, 2000, 16, 2, 128, BF), (1500, 2100, 16, 4, 64, BF), (1030, 1100, 32, 1, 256, BF), (1500, 1500, 16, 2, 64, F32),
        (1060, 1060, 20, 2, 128, F32), (1030, 1030, 16, 16, 256, F32)]


@pytest.mark.parametrize("with_lse", [False, True])
@pytest.mark.parametrize("lq,lk,hq,hk,d,dtype", BUSY)
def test_tiles_for_most_of_the_chip(lq, lk, hq, hk, d, dtype, with_lse):
    assert gdn.gdn_attn_prefill_workspace_bytes(1, lq, lk, hq, hk, d, dtype) == 0
    test_large_prefills(lq, lk, hq, hk, d, dtype, with_lse)


@pytest.mark.parametrize("lq,lk,hq,hk,d,dtype", BUSY)
@pytest.mark.parametrize("bad", [math.nan, -math.inf])
def test_bad_values_on_most_of_the_chip(lq, lk, hq, hk, d, dtype, bad):
    test_bad_values_behind_what_a_row_sees(lq, lk, hq, hk, d, dtype, bad)


@pytest.mark.parametrize("seed", range(16))
def test_random_prefills_after_contexts(seed):
    """A few new tokens after long contexts of several lengths, strided and with the heads outside."""
    r = random.Random(3000 + seed)
    dtype, d = r.choice([BF, BF, F32]), r.choice([64, 128, 256])
    hk, g, n = r.choice([1, 2, 3]), r.choice([1, 2, 5, 8]), r.randint(1, 4)
    lq = [r.choice([0, 1, r.randint(1, 90)]) for _ in range(n)] + [1]
    lk = [r.choice([0, x, r.randint(1, 3000), 2048]) for x in lq[:-1]] + [2000 * n]
    causal = r.random() < 0.8
    q, k, v = make(lq, lk, hk * g, hk, d, dtype, seed=seed)
    assert gdn.gdn_attn_prefill_workspace_bytes(n + 1, sum(lq), sum(lk), hk * g, hk, d, dtype) > 0
    kv = torch.stack([k, v], 1).to(DEV)                          # tokens, k or v, heads
    qt = q.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)  # a head's tokens together
    lse = torch.full(q.shape[:2], 5.0, device=DEV)
    out = gdn.gdn_attn_prefill(qt, kv[:, 0], kv[:, 1], ints(offsets(lq)), ints(offsets(lk)), causal=causal, lse=lse)
    compare(q, k, v, lq, lk, causal, d ** -0.5, out, lse, f"{lq} {lk}")


def test_many_sequences():
    """More sequences than a wave looks up at a time, empty ones among them."""
    r = random.Random(5)
    lq = [r.choice([0, 1, 3, 40]) for _ in range(200)]
    q, k, v = make(lq, lq, 4, 2, 64, BF)
    out, lse = run(q, k, v, lq, lq)
    compare(q, k, v, lq, lq, True, 64 ** -0.5, out, lse)
    cache = Cache(lq, 16, 2, 64, BF)
    cu, start = ints(offsets(lq)), ints([0] * 200)
    gdn.gdn_kv_write(k.to(DEV), v.to(DEV), *cache.args(), start, cu)
    kk, vv = gdn.gdn_kv_read(*cache.args(), start, cu, sum(lq))
    assert torch.equal(kk.cpu(), k) and torch.equal(vv.cpu(), v)


def test_heads_far_apart():
    """Head and token strides that put a sequence's rows beyond 32-bit byte offsets from each other."""
    d, t, h = 64, 300, 3
    far = (1 << 31) // h // 2 // 64 * 64 + 64  # elements between heads: the last lies past 2 GiB
    q, k, v = make([t], [t], h, h, d, BF)
    base = torch.zeros((h - 1) * far + t * d, dtype=BF, device=DEV)
    view = base.as_strided((t, h, d), (d, far, 1))
    view.copy_(k.to(DEV))
    out = gdn.gdn_attn_prefill(q.to(DEV), view, v.to(DEV), ints([0, t]))
    compare(q, k, v, [t], [t], True, d ** -0.5, out, None)
    wide = (1 << 22) - 64  # the largest token stride
    base = torch.zeros((t - 1) * wide + h * d, dtype=BF, device=DEV)
    view = base.as_strided((t, h, d), (wide, d, 1))
    view.copy_(v.to(DEV))
    out = gdn.gdn_attn_prefill(q.to(DEV), k.to(DEV), view, ints([0, t]))
    compare(q, k, v, [t], [t], True, d ** -0.5, out, None)
