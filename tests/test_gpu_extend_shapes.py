"""GPU: attention of new tokens over the cache over random and large shapes, so that every kernel, workgroup
shape, division of the keys and lookup of sequences runs, against a 64-bit evaluation
(tests/attn_ref.py) of all rows or a sample of them."""
import random

import pytest
import torch

import attn_ref
import gated_deltanet_linear_prefill_amd as gdn
from test_gpu_attn_decode import dense, fill
from test_gpu_attn_extend import batch, compare, queries, sight  # noqa: F401
from test_gpu_kv_cache import BF, DEV, F8, F32, Cache, ints, offsets

pytestmark = pytest.mark.gpu


def sampled(cache, q, lens_q, lens, out, lse, window, sinks, rng, rows=12, heads=3):
    """compare() of some rows and heads of every sequence, the first and the last among them."""
    g, at = q.shape[1] // cache.h, 0
    for s, (lq, length) in enumerate(zip(lens_q, lens)):
        pick = sorted({0, lq - 1, *(rng.randrange(lq) for _ in range(rows))}) if lq else []
        if pick:
            k, v, there = dense(cache, s, length)
            allowed = (sight(lq, length, window, sinks) & there[None])[pick]
            i = [at + x for x in pick]
            for h in sorted({0, q.shape[1] - 1, *(rng.randrange(q.shape[1]) for _ in range(heads))}):
                ref = attn_ref.attend(q[i, h], k[:, h // g], v[:, h // g], cache.d ** -0.5, allowed)
                attn_ref.check(out[i, h], lse[i, h], *ref, what=f"sequence {s} head {h}")
        at += lq


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(seed):
    rng = random.Random(seed)
    dtype, store = rng.choice([(BF, BF), (BF, BF), (BF, F8), (F32, F32), (F32, F8)])
    d, hk, g = rng.choice([64, 128, 256]), rng.choice([1, 2, 3]), rng.choice([1, 2, 5, 8, 17])
    n, page = rng.choice([1, 2, 5, 9]), rng.choice([16, 32, 128])
    most = rng.choice([1, 4, 20, 150])
    lens_q = [rng.randint(0, most) for _ in range(n)]
    if sum(lens_q) == 0:
        lens_q[0] = 1
    lens = [max(x + rng.choice([0, 0, 1, rng.randint(0, 900)]) - rng.choice([0, 0, 0, 1]), 0) for x in lens_q]
    window = rng.choice([0, 0, rng.randint(1, 300)])
    sinks = rng.choice([0, rng.randint(1, 60)])
    cache = Cache(lens, page, hk, d, store, seed=seed)
    fill(cache, seed, nan_behind=lens)
    q = queries(sum(lens_q), hk * g, d, dtype, seed)
    lse = torch.full(q.shape[:2], 5.0, device=DEV)
    kw = rng.choice([{}, dict(max_q=max(lens_q)), dict(max_q=max(lens_q), max_len=max(max(lens), 1))])
    out = gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints(lens), ints(offsets(lens_q)), window=window, sinks=sinks, lse=lse,
                              **kw, **cache.scales())
    sampled(cache, q, lens_q, lens, out, lse, window, sinks, rng)


@pytest.mark.parametrize("n", [64, 65, 200, 256, 257, 700])
@pytest.mark.parametrize("store,dtype", [(BF, BF), (F8, BF)])
def test_many_sequences(n, store, dtype):
    """Sequences looked up in order of length, counted, and in spread slots; many of them empty."""
    rng = random.Random(n)
    lens_q = [rng.choice([0, 0, 1, 1, 3, rng.randint(0, 90)]) for _ in range(n)]
    lens = [x + rng.randint(0, 40) for x in lens_q]
    lens_q[n // 2], lens[n // 2] = 100, 333  # rows of more than one tile
    cache = Cache(lens, 16, 1, 64, store, seed=1)
    fill(cache, 3)
    q = queries(sum(lens_q), 2, 64, dtype)
    lse = torch.full(q.shape[:2], 5.0, device=DEV)
    out = gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints(lens), ints(offsets(lens_q)), lse=lse, **cache.scales())
    compare(cache, q, lens_q, lens, out, lse, 64 ** -0.5)


LARGE = [  # rows, context, h_q, h_kv, d, store, dtype, window, sinks, tight bounds
    (4200, 300, 16, 2, 256, BF, BF, 0, 0), (4200, 9000, 16, 1, 256, BF, BF, 4000, 20), (1100, 500, 32, 8, 128, BF, BF, 0, 0),
    (1100, 3000, 32, 8, 128, BF, BF, 1000, 64), (5000, 0, 8, 8, 64, BF, BF, 0, 0), (900, 5000, 16, 2, 256, F8, BF, 0, 0),
    (2000, 100, 16, 4, 128, F8, BF, 300, 3), (700, 2000, 8, 2, 256, F32, F32, 0, 0), (3000, 100, 16, 2, 128, F32, F32, 500, 10),
    (70, 20000, 4, 1, 64, BF, BF, 0, 0), (80, 20000, 8, 1, 256, F8, BF, 0, 0), (33, 30000, 8, 1, 128, F32, F32, 0, 0),
    (600, 700, 20, 1, 64, F32, F8, 100, 7), (1, 40000, 16, 1, 256, BF, BF, 0, 0), (3, 40000, 16, 1, 64, F8, BF, 30000, 100),
]


@pytest.mark.parametrize("rows,context,hq,hk,d,store,dtype,window,sinks", LARGE)
def test_large_calls(rows, context, hq, hk, d, store, dtype, window, sinks):
    if store == F32 and dtype == F8:  # fp32 queries over an fp8 cache
        store, dtype = F8, F32
    length = rows + context
    cache = Cache([length], 64, hk, d, store)
    fill(cache, 2)
    q = queries(rows, hq, d, dtype)
    lse = torch.full(q.shape[:2], 5.0, device=DEV)
    out = gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints([length]), ints([0, rows]), window=window, sinks=sinks, lse=lse,
                              max_q=rows, max_len=length, **cache.scales())
    sampled(cache, q, [rows], [length], out, lse, window, sinks, random.Random(1), rows=20, heads=2)
    again = gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints([length]), ints([0, rows]), window=window, sinks=sinks,
                                max_q=rows, max_len=length, **cache.scales())
    same = gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints([length]), ints([0, rows]), window=window, sinks=sinks,
                               max_q=rows, max_len=length, **cache.scales())
    assert torch.equal(again, same)


@pytest.mark.parametrize("store,dtype", [(BF, BF), (F8, BF), (F32, F32)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_batch_of_both_kinds(store, dtype, d):
    """Sequences that decode beside sequences that bring hundreds of rows, ragged contexts, pages not there."""
    lens_q, lens = [1, 400, 0, 3, 1, 70, 900, 16], [2000, 900, 50, 17, 3, 1500, 900, 16]
    cache = Cache(lens, 32, 2, d, store)
    fill(cache, 2)
    for s, x in ((0, 5), (0, 40), (1, 0), (5, 30)):
        cache.table[s][x] = -1
        cache.page_table[s, x] = -1
    q = queries(sum(lens_q), 8, d, dtype)
    for window, sinks in ((0, 0), (200, 30)):
        lse = torch.full(q.shape[:2], 5.0, device=DEV)
        out = gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints(lens), ints(offsets(lens_q)), window=window, sinks=sinks, lse=lse,
                                  max_q=900, max_len=2000, **cache.scales())
        sampled(cache, q, lens_q, lens, out, lse, window, sinks, random.Random(3))


def test_lds_that_holds_nan():
    """What the kernels have not written in LDS does not reach a result."""
    lens_q, lens = [300, 5], [333, 50]
    for store, dtype, d in ((BF, BF, 128), (F8, BF, 256), (F8, BF, 64), (F32, F32, 64), (BF, BF, 256)):
        cache = Cache(lens, 16, 1, d, store)
        fill(cache, 2)
        q = queries(305, 2, d, dtype).to(DEV)
        sink = torch.zeros(1, dtype=torch.int32, device=DEV)
        gdn.debug_fill_lds(sink, blocks=1024)
        out = gdn.gdn_attn_extend(q, *cache.args(), ints(lens), ints(offsets(lens_q)), **cache.scales())
        gdn.debug_fill_lds(sink, blocks=1024)
        few = gdn.gdn_attn_extend(q[300:], *cache.args(), ints(lens), ints([0, 0, 5]), **cache.scales())
        compare(cache, q.cpu(), lens_q, lens, out, None, d ** -0.5)
        compare(cache, q[300:].cpu(), [0, 5], lens, few, None, d ** -0.5)


def test_page_ids_past_31_bits_of_rows():
    """Pages whose rows times heads pass 2^31: the last of a pool of 2^31 rows and more (fp8, one tensor
    for keys and values)."""
    if torch.cuda.mem_get_info()[0] < 180 << 30:
        pytest.skip("needs 140 GB of device memory")
    h, d, page = 8, 64, 1024
    pages = (1 << 31) // (h * page) + 3
    pool = torch.zeros(pages, h, page, d, dtype=torch.uint8, device=DEV).view(F8)
    scale = torch.full((pages, h, page), 127, dtype=torch.uint8, device=DEV)
    small = Cache([200], 1024, h, d, F8, spare=0, extra_width=0)
    fill(small, 4)
    pool.view(torch.uint8)[-1].copy_(small.k.view(torch.uint8)[0])
    scale[-1].copy_(small.ks[0])
    table = ints([[pages - 1]])
    for rows in (2, 90):
        q = queries(rows, 16, d, BF).to(DEV)
        a = gdn.gdn_attn_extend(q, pool, pool, table, ints([200]), ints([0, rows]), k_scale=scale, v_scale=scale)
        b = gdn.gdn_attn_extend(q, small.k, small.k, ints([[0]]), ints([200]), ints([0, rows]), k_scale=small.ks, v_scale=small.ks)
        assert torch.equal(a, b)
    del pool, scale
    torch.cuda.empty_cache()


@pytest.mark.parametrize("hq,hk,d,page,store,dtype", [(8, 2, 128, 16, BF, BF), (16, 2, 256, 64, F8, BF), (4, 2, 64, 32, BF, BF), (4, 1, 128, 16, F32, F32), (16, 1, 256, 16, BF, BF)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 20)])
def test_uneven_lengths_and_loose_bounds(hq, hk, d, page, store, dtype, window, sinks):
    """Few rows of sequences whose lengths are far apart, empty ones and ones without rows among them, under a
    bound on the lengths that is many times theirs, as a captured graph has it; and some tokens beyond max_q."""
    lens = [9000, 1, 0, 130, 700, 64, 2500, 17, 5000, 40, 333]
    lens_q = [2, 1, 1, 0, 5, 3, 4, 1, 1, 6, 2]
    cache = Cache(lens, page, hk, d, store, seed=2, extra_width=1 + 40000 // page)
    fill(cache, 2, nan_behind=lens)
    q = queries(sum(lens_q), hq, d, dtype)
    for max_len in (None, 9000):
        for most in (6, 4):
            lse = torch.full(q.shape[:2], 7.0, device=DEV)
            out = torch.full(q.shape, 7.0, dtype=dtype, device=DEV)
            gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints(lens), ints(offsets(lens_q)), window=window, sinks=sinks, max_q=most,
                                max_len=max_len, out=out, lse=lse, **cache.scales())
            at = 0
            for s, (m, length) in enumerate(zip(lens_q, lens)):
                done = min(m, most)
                assert bool((out[at + done:at + m] == 7.0).all()) and bool((lse[at + done:at + m] == 7.0).all())
                k, v, there = dense(cache, s, length)
                allowed = (sight(m, length, window, sinks) & there[None])[:done]
                for h in range(hq if done else 0):
                    ref = attn_ref.attend(q[at:at + done, h], k[:, h * hk // hq], v[:, h * hk // hq], d ** -0.5, allowed)
                    attn_ref.check(out[at:at + done, h], lse[at:at + done, h], *ref, what=f"sequence {s} head {h}")
                at += m


def test_offsets_that_go_back():
    """Offsets that decrease or lie past the tokens give their sequences no rows or fewer; the others are right."""
    lens = [3000, 200, 900, 50]
    cache = Cache(lens, 16, 2, 128, BF)
    fill(cache, 3)
    q = queries(12, 8, 128, BF)
    out = gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints(lens), ints([0, 4, 2, 9, 4000]), max_q=8)
    compare(cache, q, [2], [2998], out[:2], None, 128 ** -0.5)  # rows 2 and 3 are two sequences'
    k, v, _ = dense(cache, 2, 900)
    allowed = sight(7, 900, 0, 0)[2:]
    for h in range(8):
        attn_ref.check(out[4:9, h], None, *attn_ref.attend(q[4:9, h], k[:, h // 4], v[:, h // 4], 128 ** -0.5, allowed), what=f"head {h}")
    k, v, _ = dense(cache, 3, 50)
    for h in range(8):
        attn_ref.check(out[9:, h], None, *attn_ref.attend(q[9:, h], k[:, h // 4], v[:, h // 4], 128 ** -0.5, sight(3, 50, 0, 0)), what=f"head {h}")


@pytest.mark.parametrize("dtype,store", [(BF, BF), (BF, F8), (F32, F32), (F32, F8)])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens_q,lens,hq,hk", [([7], [900], 4, 1), ([3, 5, 0, 6], [700, 5, 40, 1500], 8, 2), ([16, 9], [600, 130], 8, 2), ([13, 1, 16], [13, 900, 17], 4, 1)])
def test_larger_tiles_of_few_rows(lens_q, lens, hq, hk, d, dtype, store):
    """17 to 64 rows of a KV head under bounds that ask for much reading: tiles of 32 and 64 rows, whole and in part,
    with and without a window; under tight bounds the tiles are of 16 rows."""
    cache = Cache(lens, 16, hk, d, store, seed=4, extra_width=200000)
    fill(cache, 4, nan_behind=None)
    q = queries(sum(lens_q), hq, d, dtype)
    for window, sinks in ((0, 0), (1000000, 3)):
        lse = torch.zeros(q.shape[:2], device=DEV)
        for max_len in (None, max(lens)):
            out = gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints(lens), ints(offsets(lens_q)), max_q=max(lens_q), max_len=max_len, window=window,
                                      sinks=sinks, lse=lse, **cache.scales())
            compare(cache, q, lens_q, lens, out, lse, d ** -0.5, window, sinks)


@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 4)])
def test_more_sequences_than_lanes_with_drafts(window, sinks):
    """fp8 pages with d = 256 and 70 sequences: tiles of 32 rows, in slots that are not divided by lengths."""
    rng = random.Random(5)
    lens_q = [rng.choice((0, 1, 3, 5, 8)) for _ in range(70)]
    lens = [rng.choice((0, 1, 40, 300)) + m for m in lens_q]
    cache = Cache(lens, 16, 1, 256, F8, seed=4)
    fill(cache, 4, nan_behind=lens)
    q = queries(sum(lens_q), 6, 256, BF)
    lse = torch.zeros(q.shape[:2], device=DEV)
    out = gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints(lens), ints(offsets(lens_q)), max_q=8, window=window, sinks=sinks, lse=lse, **cache.scales())
    compare(cache, q, lens_q, lens, out, lse, 256 ** -0.5, window, sinks)
